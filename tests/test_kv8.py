"""The 8-bit cache's host side (no GPU): refused arguments, workspace sizes, and
the definitions themselves."""

import ctypes
import math

import pytest
import torch

import kv8_plain as P
from flow_matching_dit_cosmot_b200 import _lib as L
from flow_matching_dit_cosmot_b200 import api as A


def cache(**kw):
    f = dict(k=256, v=512, k_scale=1024, v_scale=2048, lens=4096, ld=256, batch_stride=100, batch=2, capacity=100,
             n_kv_heads=2, head_dim=128, block=64, reserved=0)
    f.update(kw)
    return L.Kv8Cache(**f)


def query(**kw):
    f = dict(n_q=3, q_batch_stride=3, o_batch_stride=3, n_heads=4, n_new=0, mask_mode=0, max_len=0, softmax_scale=0.0)
    f.update(kw)
    return L.Kv8Query(**f)


BAD_CACHES = [
    (dict(head_dim=96), L.COSMOT_ERR_UNSUPPORTED), (dict(block=8), L.COSMOT_ERR_UNSUPPORTED),
    (dict(block=48), L.COSMOT_ERR_UNSUPPORTED), (dict(k=0), L.COSMOT_ERR_INVALID_ARG),
    (dict(v_scale=0), L.COSMOT_ERR_INVALID_ARG), (dict(lens=0), L.COSMOT_ERR_INVALID_ARG),
    (dict(k=260), L.COSMOT_ERR_INVALID_ARG), (dict(ld=248), L.COSMOT_ERR_INVALID_ARG),
    (dict(ld=264), L.COSMOT_ERR_INVALID_ARG), (dict(batch_stride=99), L.COSMOT_ERR_INVALID_ARG),
    (dict(capacity=0), L.COSMOT_ERR_INVALID_ARG), (dict(batch=0), L.COSMOT_ERR_INVALID_ARG),
    (dict(batch=40_000), L.COSMOT_ERR_UNSUPPORTED), (dict(capacity=2 ** 31 - 1, batch=1), L.COSMOT_ERR_UNSUPPORTED),
    (dict(batch_stride=2 ** 31), L.COSMOT_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(change, want):
    lib = L.lib()
    c, q, n = ctypes.byref(cache(**change)), ctypes.byref(query()), ctypes.c_size_t(0)
    assert lib.cosmot_kv8_store(c, 256, 256, 256, 4, 4, None) == want
    assert lib.cosmot_kv8_attention_workspace(c, q, ctypes.byref(n)) == want
    assert lib.cosmot_kv8_attention(c, q, 256, 512, 256, 512, None, None, 0, None) == want
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, 256, 1.0, 256, None) == want
    assert lib.cosmot_kv8_evict_workspace(c, ctypes.byref(n)) == want
    assert lib.cosmot_kv8_evict(c, 256, 4, 0, 0, 256, 256, 256, 1 << 20, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n_heads=3), L.COSMOT_ERR_INVALID_ARG), (dict(n_heads=0), L.COSMOT_ERR_INVALID_ARG),
    (dict(n_q=-1), L.COSMOT_ERR_INVALID_ARG), (dict(n_new=-1), L.COSMOT_ERR_INVALID_ARG),
    (dict(n_new=101), L.COSMOT_ERR_INVALID_ARG), (dict(mask_mode=2), L.COSMOT_ERR_INVALID_ARG),
    (dict(max_len=-1), L.COSMOT_ERR_INVALID_ARG), (dict(q_batch_stride=2), L.COSMOT_ERR_INVALID_ARG),
    (dict(o_batch_stride=2), L.COSMOT_ERR_INVALID_ARG), (dict(softmax_scale=-1.0), L.COSMOT_ERR_INVALID_ARG),
    (dict(softmax_scale=math.nan), L.COSMOT_ERR_INVALID_ARG), (dict(softmax_scale=math.inf), L.COSMOT_ERR_INVALID_ARG),
    (dict(n_q=2 ** 31, q_batch_stride=2 ** 31, o_batch_stride=2 ** 31), L.COSMOT_ERR_UNSUPPORTED)])
def test_bad_queries_are_refused(change, want):
    lib = L.lib()
    c, q, n = ctypes.byref(cache()), ctypes.byref(query(**change)), ctypes.c_size_t(0)
    assert lib.cosmot_kv8_attention_workspace(c, q, ctypes.byref(n)) == want
    assert lib.cosmot_kv8_attention(c, q, 256, 512, 256, 512, None, 256, 1 << 30, None) == want
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, 256, 1.0, 256, None) == want


def test_bad_pointers_strides_and_workspaces_are_refused():
    lib, bad = L.lib(), L.COSMOT_ERR_INVALID_ARG
    c, q = ctypes.byref(cache()), ctypes.byref(query())
    assert lib.cosmot_kv8_store(None, 256, 256, 256, 4, 4, None) == bad
    assert lib.cosmot_kv8_store(c, None, 256, 256, 4, 4, None) == bad
    assert lib.cosmot_kv8_store(c, 264, 256, 256, 4, 4, None) == bad       # not 16-byte aligned
    assert lib.cosmot_kv8_store(c, 256, 256, 252, 4, 4, None) == bad       # rows overlap
    assert lib.cosmot_kv8_store(c, 256, 256, 260, 4, 4, None) == bad       # ld % 8
    assert lib.cosmot_kv8_store(c, 256, 256, 256, 3, 4, None) == bad       # sequences overlap
    assert lib.cosmot_kv8_store(c, 256, 256, 256, 4, -1, None) == bad
    assert lib.cosmot_kv8_store(c, 256, 256, 256, 101, 101, None) == bad   # more rows than the capacity
    assert lib.cosmot_kv8_store(c, 256, 256, 256, 4, 0, None) == L.COSMOT_OK
    assert lib.cosmot_kv8_attention(c, None, 256, 512, 256, 512, None, None, 0, None) == bad
    assert lib.cosmot_kv8_attention(c, q, None, 512, 256, 512, None, None, 0, None) == bad
    assert lib.cosmot_kv8_attention(c, q, 256, 504, 256, 512, None, None, 0, None) == bad
    assert lib.cosmot_kv8_attention(c, q, 256, 512, 264, 512, None, None, 0, None) == bad
    assert lib.cosmot_kv8_attention(c, q, 256, 512, 256, 504, None, None, 0, None) == bad
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, None, 1.0, 256, None) == bad
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, 256, 1.0, None, None) == bad
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, 256, -0.5, 256, None) == bad
    assert lib.cosmot_kv8_weigh(c, q, 256, 512, 256, math.nan, 256, None) == bad
    n = L.cosmot_kv8_evict_workspace(cache())
    assert n >= 2 * 2 * 2 * 4
    for a in ((None, 4, 0, 0, 256, 256, 256, n), (256, 0, 0, 0, 256, 256, 256, n), (256, 4, -1, 0, 256, 256, 256, n),
              (256, 4, 0, -1, 256, 256, 256, n), (256, 4, 0, 0, None, 256, 256, n), (256, 4, 0, 0, 256, None, 256, n),
              (256, 4, 0, 0, 256, 256, None, n), (256, 4, 0, 0, 256, 256, 272, n)):
        assert lib.cosmot_kv8_evict(c, *a, None) == bad
    assert lib.cosmot_kv8_evict(c, 256, 4, 0, 0, 256, 256, 256, n - 1, None) == L.COSMOT_ERR_WORKSPACE
    # a call whose keys are split needs its workspace
    long = cache(capacity=100_000, batch_stride=100_000)
    need = L.cosmot_kv8_attention_workspace(long, query())
    assert need > 0
    args = (ctypes.byref(long), q, 256, 512, 256, 512, None)
    assert lib.cosmot_kv8_attention(*args, None, 0, None) == bad
    assert lib.cosmot_kv8_attention(*args, 272, need, None) == bad
    assert lib.cosmot_kv8_attention(*args, 256, need - 1, None) == L.COSMOT_ERR_WORKSPACE
    # no queries: nothing to do
    assert lib.cosmot_kv8_attention(c, ctypes.byref(query(n_q=0)), 256, 512, 256, 512, None, None, 0, None) == L.COSMOT_OK


@pytest.mark.parametrize("n_q,heads,capacity", [(1, 4, 100_000), (40, 2, 9_000), (1560, 2, 20_000), (573, 8, 100_000)])
def test_a_split_call_needs_its_workspace(n_q, heads, capacity):
    """Few rows and tiles; the bytes do not shrink with the bound on the lengths
    being given up (0: the capacity), and too few are refused."""
    lib = L.lib()
    c = cache(capacity=capacity, batch_stride=capacity, batch=1)
    kw = dict(n_q=n_q, q_batch_stride=n_q, o_batch_stride=n_q, n_heads=heads)
    need = L.cosmot_kv8_attention_workspace(c, query(**kw))
    assert need > 0 and need >= L.cosmot_kv8_attention_workspace(c, query(**kw, max_len=64))
    assert L.cosmot_kv8_attention_workspace(c, query(**kw, max_len=capacity)) == need
    assert L.cosmot_kv8_attention_workspace(c, query(**kw, max_len=2 ** 31 - 1)) == need
    ld = heads * 128
    args = (ctypes.byref(c), ctypes.byref(query(**kw)), 256, ld, 256, ld, None)
    assert lib.cosmot_kv8_attention(*args, None, need, None) == L.COSMOT_ERR_INVALID_ARG
    assert lib.cosmot_kv8_attention(*args, 256, need - 1, None) == L.COSMOT_ERR_WORKSPACE
    assert L.cosmot_kv8_attention_workspace(c, query(**{**kw, "n_q": 0})) == 0


def test_the_python_layer_refuses_cpu_tensors_and_bad_layouts():
    t = torch.zeros((1, 16, 1, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((1, 1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        A.KVCache8(t, t, s, s, torch.zeros(1, dtype=torch.int32), 16)
    f = A._rows_layout
    x = torch.zeros((2, 5, 6, 64), dtype=torch.bfloat16)
    assert f(x[:, :, 2:4], "x", 2, 2, 64, torch.bfloat16) == (384, 5)
    assert f(x[:, :3, 2:4], "x", 2, 2, 64, torch.bfloat16) == (384, 5)
    assert f(x[:, :1], "x", 2, 6, 64, torch.bfloat16) == (5 * 384, 1)
    assert f(x[:1, :1], "x", 1, 6, 64, torch.bfloat16) == (384, 1)
    for bad in (x[:, :, ::2], x[:, ::2], x.transpose(1, 2), x[:1].expand(2, 5, 6, 64), x[:, :1].expand(2, 5, 6, 64), x[..., :32],
                x.float(), x[0]):
        with pytest.raises(ValueError):
            f(bad, "x", 2, None, 64, torch.bfloat16)


def test_the_definitions():
    """e4m3 rounding against torch's conversion; the scale rule at its borders;
    the softmax against torch's in 64 bits."""
    y = torch.cat([torch.linspace(-448, 448, 20_001), torch.linspace(-0.04, 0.04, 8_001)]).float()
    assert torch.equal(P.nearest8(y.double()).float(), y.to(torch.float8_e4m3fn).float())
    assert P.scale_of(448.0) == 1.0 and P.scale_of(448.0 * (1 + 2 ** -8)) == 2.0 and P.scale_of(224.0) == 0.5
    assert P.scale_of(0.0) == 2.0 ** -40 and P.scale_of(1e38) == 2.0 ** 40
    gen = torch.Generator().manual_seed(0)
    q = torch.randn((1, 5, 2, 64), generator=gen, dtype=torch.float64)
    K, V = (torch.randn((1, 9, 1, 64), generator=gen, dtype=torch.float64) for _ in range(2))
    o, lse, *_ = P.attend(q, K, V, [9], True)
    s = torch.einsum("bqhd,bkd->bhqk", q, K[:, :, 0]) / 8
    s = s.masked_fill(torch.arange(9) > torch.arange(5)[:, None] + 4, -math.inf)
    torch.testing.assert_close(lse, torch.logsumexp(s, -1))
    torch.testing.assert_close(o, torch.einsum("bhqk,bkd->bqhd", s.softmax(-1), V[:, :, 0]))
    w, _ = P.weigh(q, K, lse, [9], 4, True, torch.zeros((1, 1, 3)), 1.0)
    torch.testing.assert_close(w.sum(), torch.tensor(10.0, dtype=torch.float64))

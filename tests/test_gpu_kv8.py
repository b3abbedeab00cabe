"""The 8-bit key/value cache on the GPU against its definitions in 64 bits."""

import math

import pytest
import torch

import kv8_plain as P
from gpu_helpers import assert_device_ok

pytestmark = pytest.mark.gpu

from flow_matching_dit_cosmot_b200 import _lib as L  # noqa: E402
from flow_matching_dit_cosmot_b200 import api as A  # noqa: E402

F8 = torch.float8_e4m3fn


def rows(seed, *shape, spread=0.5):
    """bf16 rows with channels (and heads) of different size."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * torch.exp(spread * torch.randn(shape[2:], generator=gen, device="cuda"))).to(torch.bfloat16)


def filled(batch, cap, g, hd, block, lens, seed=0, spread=0.5):
    """A cache whose sequences hold lens rows; the bytes behind them are NaN, and so are the scales of the blocks
    that hold no row: nothing may read them."""
    c = A.KVCache8.empty(batch, cap, g, hd, block)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7f)
    for t in (c.k_scale, c.v_scale):
        t.fill_(math.nan)
    top = max(lens)
    if top:
        k, v = rows(seed + 1, batch, top, g, hd, spread=spread), rows(seed + 2, batch, top, g, hd, spread=spread)
        for src, dst, sc in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
            val = torch.zeros((batch, cap, g, hd), dtype=torch.float64)
            s = torch.ones(sc.shape, dtype=torch.float64)
            P.store(val, s, [0] * batch, src.double().cpu(), block)
            for b, n in enumerate(lens):
                dst[b, :n] = val[b, :n].to(torch.float32).to(F8).cuda()
                nb = -(-n // block)
                sc[b, :, :nb] = s[b, :, :nb].float().cuda()
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return c


def dequant(c, lens):
    """Float64 values with zeros behind the rows held."""
    out = []
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = P.values(t, s, c.block)
        for b, n in enumerate(lens):
            x[b, n:] = 0
        out.append(x)
    return out


def queries(seed, batch, n, H, hd, g=None):
    """bf16 queries as the leading columns of a QKV projection's rows."""
    gen = torch.Generator("cuda").manual_seed(seed)
    wide = torch.randn((batch, n, H + (2 * g if g else 0), hd), generator=gen, device="cuda") * 1.5
    return wide.to(torch.bfloat16)[:, :, :H]


def check_attend(c, q, lens, causal, n_new=0, scale=None, **kw):
    shown = [n + n_new for n in lens]
    K, V = dequant(c, shown)
    o, lse = c.attend(q, n_new=n_new, causal=causal, softmax_scale=scale or 0.0, **kw)
    torch.cuda.synchronize()
    assert_device_ok()
    ro, rl, bo, bl, _ = P.attend(q, K, V, shown, causal, scale)
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none) and bool((lse[none] < 0).all())
    el = torch.where(none, 0.0, (lse.double() - rl).abs())
    assert bool((el <= bl).all()), f"lse: {float((el - bl).max()):.3g} over its bound"
    eo = (o.double() - ro).abs()
    assert bool(torch.isfinite(o).all())
    print(f"[kv8] o: worst error / bound {float((eo / bo.clamp(min=1e-300)).max()):.2f}, lse {float((el / bl.clamp(min=1e-300)).max()):.2f}")
    assert bool((eo <= bo).all()), f"o: {float((eo - bo).max()):.3g} over its bound"
    return o, lse


def check_weigh(c, q, lse, lens, causal, n_new=0, decay=0.75, scale=None):
    shown = [n + n_new for n in lens]
    K, _ = dequant(c, shown)
    gen = torch.Generator("cuda").manual_seed(9)
    w = torch.rand((c.batch, c.n_kv_heads, c.n_blocks), generator=gen, device="cuda")
    ref, bound = P.weigh(q, K, lse, shown, c.block, causal, w, decay, scale)
    before = w.clone()
    c.weigh(q, lse, w, decay=decay, n_new=n_new, causal=causal, softmax_scale=scale or 0.0)
    torch.cuda.synchronize()
    assert_device_ok()
    err = (w.double() - ref).abs()
    print(f"[kv8] weight: worst error / bound {float((err / bound.clamp(min=1e-300)).max()):.2f}")
    assert bool((err <= bound).all()), f"weight: {float((err - bound).max()):.3g} over its bound"
    for b, n in enumerate(shown):
        nb = -(-n // c.block)
        assert torch.equal(w[b, :, nb:], before[b, :, nb:])


# ------------------------------------------------------------------ store

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,n", [([0], 1), ([0, 0], 300), ([5, 130, 63], 1), ([17, 0, 200], 77), ([128, 127, 129], 128)])
def test_store_matches_the_definition_bit_for_bit(hd, block, lens, n):
    B, g, cap = len(lens), 3, max(lens) + n + 5
    c = filled(B, cap, g, hd, block, lens, seed=3)
    wide = rows(7, B, n, 2 + 2 * g, hd, spread=1.5) * 4  # some first blocks get a larger scale, some keep theirs
    k, v = wide[:, :, 2:2 + g], wide[:, :, 2 + g:]
    want = []
    for t, s, x in ((c.k, c.k_scale, k), (c.v, c.v_scale, v)):
        val, sc = t.double().cpu(), s.double().cpu()
        P.store(val, sc, lens, x.double().cpu(), block)
        want.append((val, sc))
    c.store(k, v)
    torch.cuda.synchronize()
    assert_device_ok()
    for (val, sc), t, s in zip(want, (c.k, c.v), (c.k_scale, c.v_scale)):
        torch.testing.assert_close(t.double().cpu(), val, rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(s.double().cpu(), sc, rtol=0, atol=0, equal_nan=True)


def test_store_special_values():
    """Zeros, subnormals, infinities, NaN and magnitudes beyond the scale's range."""
    x = torch.zeros((1, 128, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0:16] = 0
    x[0, 16, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3.5])
    x[0, 32, 0, :3] = torch.tensor([1e38, -2e37, 1.0])       # beyond 448 * 2^40: saturates
    x[0, 48, 0, :3] = torch.tensor([1e-30, -1e-20, 0.0])     # below 2^-40's smallest step: zero
    x[0, 64, 0, :3] = torch.tensor([448.0, 449.0 * 1.01, -0.0])
    x[0, 80, 0, :2] = torch.tensor([math.inf, math.nan])     # nothing finite but zeros
    c = A.KVCache8.empty(1, 128, 1, 64, 16)
    val, sc = c.k.double().cpu(), c.k_scale.double().cpu()
    P.store(val, sc, [0], x.double().cpu(), 16)
    c.store(x, x)
    torch.cuda.synchronize()
    torch.testing.assert_close(c.k.double().cpu(), val, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(c.v_scale.double().cpu(), sc)
    assert sc[0, 0, 0] == 2.0 ** -40 and sc[0, 0, 2] == 2.0 ** 40 and sc[0, 0, 5] == 2.0 ** -40


def test_store_again_over_the_same_rows_is_the_same():
    """A denoising step stores its block anew: same rows in, same cache out."""
    c = filled(2, 200, 2, 64, 64, [70, 3], seed=5)
    k, v = rows(1, 2, 60, 2, 64) * 8, rows(2, 2, 60, 2, 64)
    c.store(k, v)
    first = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    c.store(k, v)
    for a, b in zip(first, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_length_without_room_is_reported_and_nothing_is_written():
    c = filled(2, 64, 2, 64, 16, [60, 10], seed=6)
    before = c.k.view(torch.uint8).clone()
    x = rows(1, 2, 8, 2, 64)
    c.store(x, x)
    torch.cuda.synchronize()
    st, where = L.cosmot_get_device_status(torch.cuda.current_stream().cuda_stream)
    assert (st, where) == (L.COSMOT_ERR_BOUNDS, 400)
    assert torch.equal(before[0], c.k.view(torch.uint8)[0])
    assert not torch.equal(before[1, 10:18], c.k.view(torch.uint8)[1, 10:18])
    for bad in (-3, 65, 2 ** 31 - 1):
        c.lens[0] = bad
        o, _ = c.attend(queries(1, 2, 1, 2, 64))
        torch.cuda.synchronize()
        assert L.cosmot_get_device_status(torch.cuda.current_stream().cuda_stream)[0] == L.COSMOT_ERR_BOUNDS
    assert_device_ok()


# ------------------------------------------------------------------ attend and weigh

SHAPES = [  # batch lengths, n_q, kv heads, group, head_dim, block, causal
    ([1], 1, 1, 1, 64, 16, False),
    ([0, 1, 15, 16, 17], 1, 2, 4, 128, 16, True),
    ([34], 34, 4, 1, 64, 16, True),
    ([500, 3, 0, 77], 7, 2, 3, 128, 64, True),      # rows that see nothing
    ([257, 640], 5, 2, 8, 64, 32, False),
    ([1023], 1, 8, 8, 128, 128, False),
    ([129, 130], 33, 3, 5, 128, 32, False),
    ([300, 260], 130, 2, 2, 64, 128, True),
    ([703, 650], 260, 2, 4, 128, 64, False),
    ([333, 12], 258, 1, 1, 128, 16, True),
    ([1200], 300, 4, 1, 128, 128, False),
    ([2000], 17, 1, 16, 64, 64, False),
]


@pytest.mark.parametrize("lens,n,g,group,hd,block,causal", SHAPES)
def test_attend_and_weigh(lens, n, g, group, hd, block, causal):
    c = filled(len(lens), max(lens) + 3, g, hd, block, lens, seed=11)
    q = queries(21, len(lens), n, g * group, hd, g)
    _, lse = check_attend(c, q, lens, causal)
    check_weigh(c, q, lse, lens, causal)


@pytest.mark.parametrize("n", [1, 40, 200])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_stored_but_not_advanced_over(n, causal):
    lens = [90, 0, 33]
    c = filled(3, 90 + n, 2, 128, 32, lens, seed=12)
    k, v = rows(31, 3, n, 2, 128), rows(32, 3, n, 2, 128)
    c.store(k, v)
    q = queries(22, 3, n, 4, 128)
    _, lse = check_attend(c, q, lens, causal, n_new=n, max_len=90 + n)
    check_weigh(c, q, lse, lens, causal, n_new=n)


@pytest.mark.parametrize("n", [1, 150])
def test_a_long_history_is_split_the_same_way_whatever_the_bound(n):
    """max_len only sizes the split: too small, too large and none give the result."""
    lens = [4500]
    c = filled(1, 4500, 1, 128, 64, lens, seed=13)
    q = queries(23, 1, n, 4, 128)
    for m in (0, 1, 600, 4500):
        check_attend(c, q, lens, False, max_len=m)


@pytest.mark.parametrize("n", [1, 64])
def test_sharp_and_flat_softmax(n):
    """Scores of +-200 (one key takes all) and all equal; a scale of the caller's."""
    lens = [700, 41]
    c = filled(2, 700, 2, 64, 32, lens, seed=14)
    q = queries(24, 2, n, 4, 64)
    _, lse = check_attend(c, q, lens, False, scale=6.0)
    check_weigh(c, q, lse, lens, False, scale=6.0)
    _, lse = check_attend(c, q * 0, lens, True)
    check_weigh(c, q * 0, lse, lens, True)


@pytest.mark.parametrize("n", [2, 140])
def test_blocks_of_very_different_scales(n):
    """Value blocks 2^30 apart, all-zero blocks, a query of large and small channels."""
    lens = [400]
    c = filled(1, 400, 1, 128, 64, lens, seed=15)
    c.v_scale[0, 0, 1] *= 2.0 ** 12
    c.v_scale[0, 0, 2] *= 2.0 ** -18
    c.v.view(torch.uint8)[0, 192:256] = 0
    c.v_scale[0, 0, 3] = 2.0 ** -40
    c.k.view(torch.uint8)[0, 256:320] = 0
    c.k_scale[0, 0, 4] = 2.0 ** -40
    c.v_scale[0, 0, 5] *= 1.37  # scales need not be powers of two
    c.k_scale[0, 0, 5] *= 0.61
    q = queries(25, 1, n, 2, 128)
    q[..., 3] *= 64
    check_attend(c, q, lens, False)


def test_a_query_that_is_not_finite_gives_nan_and_no_other_row_changes():
    lens = [150]
    c = filled(1, 150, 1, 64, 16, lens, seed=16)
    for n in (4, 200):
        q = queries(26, 1, n, 2, 64)
        good, glse = c.attend(q)
        q[0, 1, 0, 5] = math.inf
        q[0, 2, 1, 7] = math.nan
        o, lse = c.attend(q)
        bad = torch.zeros((1, n, 2), dtype=torch.bool, device="cuda")
        bad[0, 1, 0] = bad[0, 2, 1] = True
        assert bool(torch.isnan(o[bad]).all()) and bool(torch.isnan(lse.transpose(1, 2)[bad]).all())
        assert torch.equal(o[~bad], good[~bad])
        assert torch.equal(lse.transpose(1, 2)[~bad], glse.transpose(1, 2)[~bad])


@pytest.mark.parametrize("n", [1, 50, 140])
def test_outputs_stay_inside_their_rows(n):
    """A strided output with guard columns, rows and sequences."""
    lens = [77, 140]
    c = filled(2, 140, 2, 64, 16, lens, seed=17)
    q = queries(27, 2, n, 4, 64)
    raw = torch.full((3, n + 2, 6, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    out = raw[:2, :n, 1:5]
    want, _ = c.attend(q)
    c.attend(q, out=out)
    assert torch.equal(out, want)
    raw[:2, :n, 1:5] = -7.0
    assert bool((raw == -7.0).all())


@pytest.mark.parametrize("n", [1, 130])
def test_rows_far_behind_each_other(n):
    """Sequences more than 2^32 bytes apart."""
    g, hd, block, cap = 1, 128, 64, 320
    between = 36_000_000  # rows of 128 bytes
    store = torch.empty(((between + cap) * g * hd,), dtype=torch.uint8, device="cuda").view(F8)
    far = lambda: store.as_strided((2, cap, g, hd), (between * g * hd, g * hd, hd, 1))  # noqa: E731
    near = filled(2, cap, g, hd, block, [300, 211], seed=18)
    c = A.KVCache8(far(), torch.empty_like(store).as_strided((2, cap, g, hd), (between * g * hd, g * hd, hd, 1)),
                   near.k_scale.clone(), near.v_scale.clone(), near.lens, block)
    for a, b in ((c.k, near.k), (c.v, near.v)):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    q = queries(28, 2, n, 2, hd)
    o, lse = near.attend(q)
    of, lf = c.attend(q)
    assert torch.equal(o, of) and torch.equal(lse, lf)
    w, wf = near.empty_weight(), near.empty_weight()
    near.weigh(q, lse, w)
    c.weigh(q, lse, wf)
    assert torch.equal(w, wf)
    x = rows(3, 2, 20, g, hd)
    near.store(x, x)
    c.store(x, x)
    near.evict(w, 3)
    c.lens.copy_(torch.tensor([300, 211], dtype=torch.int32))
    c.evict(wf, 3)
    assert torch.equal(near.k.view(torch.uint8), c.k.view(torch.uint8))
    assert torch.equal(near.v.view(torch.uint8), c.v.view(torch.uint8))
    assert_device_ok()


# ------------------------------------------------------------------ evict

@pytest.mark.parametrize("hd,block", [(64, 16), (128, 64), (128, 128), (64, 32)])
@pytest.mark.parametrize("lens,keep,first,last", [
    ([1000, 999, 5, 0], 5, 0, 0), ([640, 640], 4, 66, 100), ([130, 700], 1, 0, 0), ([700, 130, 64], 3, 10_000, 0),
    ([512, 300], 40, 0, 1), ([2000], 9, 66, 300)])
def test_evict_matches_the_definition_bit_for_bit(hd, block, lens, keep, first, last):
    B, g = len(lens), 3
    c = filled(B, max(lens) + 7, g, hd, block, lens, seed=41)
    gen = torch.Generator("cuda").manual_seed(42)
    w = torch.rand((B, g, c.n_blocks), generator=gen, device="cuda")
    w[w < 0.3] = 0.0       # ties: the lower index stays
    w[:, 0, ::5] = 0.75
    w[:, 1, 3:6] = math.nan
    w[:, 2, 2:4] = math.inf
    w[:, 1, :2] = -0.0
    kb, vb, ks, vs = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu(), c.k_scale.cpu(), c.v_scale.cpu()
    wref, lref = P.evict(kb, vb, ks, vs, w.cpu(), lens, block, keep, first, last)
    w0 = w.clone()
    wo, lo = c.evict(w, keep, first, last, in_place=False)
    torch.cuda.synchronize()
    assert_device_ok()
    assert lo.tolist() == lref and c.lens.tolist() == lens
    assert torch.equal(w0.view(torch.int32), w.view(torch.int32))
    assert torch.equal(c.k.view(torch.uint8).cpu(), kb) and torch.equal(c.v.view(torch.uint8).cpu(), vb)
    for got, ref in ((c.k_scale, ks), (c.v_scale, vs), (wo, wref)):
        torch.testing.assert_close(got.cpu(), ref, rtol=0, atol=0, equal_nan=True)


def test_evict_in_place_is_the_same():
    lens = [900, 411]
    cs = [filled(2, 900, 2, 64, 32, lens, seed=43) for _ in range(2)]
    w = [torch.rand((2, 2, cs[0].n_blocks), generator=torch.Generator("cuda").manual_seed(5), device="cuda") for _ in cs]
    wo, lo = cs[0].evict(w[0], 8, 66, 40, in_place=False)
    wi, li = cs[1].evict(w[1], 8, 66, 40)
    assert li.data_ptr() == cs[1].lens.data_ptr() and wi.data_ptr() == w[1].data_ptr()
    assert torch.equal(wo, wi) and torch.equal(lo, li)
    assert torch.equal(cs[0].k.view(torch.uint8), cs[1].k.view(torch.uint8))
    assert torch.equal(cs[0].k_scale.nan_to_num(), cs[1].k_scale.nan_to_num())


def test_evict_again_and_again_is_the_same():
    """The moves start while the selection before them still runs: they must wait for what it writes."""
    lens = [300, 211]
    ref = None
    for k in range(40):
        c = filled(2, 320, 1, 128, 64, lens, seed=44)
        w = torch.rand((2, 1, c.n_blocks), generator=torch.Generator("cuda").manual_seed(7), device="cuda")
        junk = torch.full((1 << 16,), 0xc0 + k % 8, dtype=torch.uint8, device="cuda")  # what the workspace may hold before
        del junk
        c.evict(w, 3)
        got = (c.lens, w, c.k_scale.nan_to_num(), c.k.view(torch.uint8), c.v.view(torch.uint8))
        if ref is None:
            ref = got
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_evict_many_blocks():
    """More blocks than a CTA's threads, most of them equal."""
    lens = [60_000]
    c = A.KVCache8.empty(1, 60_000, 1, 64, 16)
    gen = torch.Generator("cuda").manual_seed(6)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 120, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
    c.lens.fill_(lens[0])
    w = (torch.rand((1, 1, c.n_blocks), generator=gen, device="cuda") * 8).floor()
    kb, vb, ks, vs = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu(), c.k_scale.cpu(), c.v_scale.cpu()
    wref, lref = P.evict(kb, vb, ks, vs, w.cpu(), lens, 16, 1717, 66, 1000)
    c.evict(w, 1717, 66, 1000)
    torch.cuda.synchronize()
    assert c.lens.tolist() == lref and torch.equal(w.cpu(), wref)
    assert torch.equal(c.k.view(torch.uint8).cpu(), kb) and torch.equal(c.v.view(torch.uint8).cpu(), vb)


# ------------------------------------------------------------------ together, streams, graphs

def _step(c, x, w, n, keep):
    """One streaming step: store, attend, weigh, advance, evict."""
    qkv = x["qkv"]
    H = qkv.shape[2] - 2 * c.n_kv_heads
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + c.n_kv_heads], qkv[:, :, H + c.n_kv_heads:]
    c.store(k, v)
    o, lse = c.attend(q, n_new=n)
    c.weigh(q, lse, w, decay=0.9, n_new=n)
    c.advance(n)
    c.evict(w, keep, first_rows=10, last_rows=n)
    return o, lse


@pytest.mark.parametrize("n", [1, 48, 150])
def test_a_rollout_with_eviction(n):
    """Store, attend, weigh and evict over many steps, against the definitions run
    alongside (the definitions evict by the kernels' weights, which the weigh
    check holds to their bound, so that both keep the same blocks)."""
    g, group, hd, block, keep, B = 2, 2, 64, 16, 14, 2
    c = filled(B, keep * block + 2 * n + 64, g, hd, block, [40, 23], seed=51)
    w = c.empty_weight()
    lens = [40, 23]
    for t in range(5):
        qkv = rows(60 + t, B, n, (group + 2) * g, hd)
        H = group * g
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + g], qkv[:, :, H + g:]
        c.store(k, v)
        _, lse = check_attend(c, q, lens, False, n_new=n)
        K, _ = dequant(c, [a + n for a in lens])
        ref, bound = P.weigh(q, K, lse, [a + n for a in lens], block, False, w, 0.9)
        c.weigh(q, lse, w, decay=0.9, n_new=n)
        assert bool(((w.double() - ref).abs() <= bound).all())
        c.advance(n)
        lens = [a + n for a in lens]
        kb, vb, ks, vs = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu(), c.k_scale.cpu(), c.v_scale.cpu()
        wref, lens = P.evict(kb, vb, ks, vs, w.cpu(), lens, block, keep, 10, n)
        c.evict(w, keep, first_rows=10, last_rows=n)
        torch.cuda.synchronize()
        assert c.lens.tolist() == lens and torch.equal(w.cpu(), wref)
        assert torch.equal(c.k.view(torch.uint8).cpu(), kb)
    assert_device_ok()


@pytest.mark.parametrize("n", [1, 150])
def test_a_captured_step_follows_the_lengths(n):
    """One graph of a whole step, replayed, equals the calls one by one; two
    graphs whose workspaces come from one pool do not disturb each other."""
    g, hd, block, keep = 2, 64, 16, 20
    make = lambda: filled(1, 900, g, hd, block, [300], seed=61)  # noqa: E731
    a, b, d = make(), make(), make()
    wa, wb, wd = a.empty_weight(), b.empty_weight(), d.empty_weight()
    x = {"qkv": rows(70, 1, n, 4 + 2 * g, hd)}
    _step(make(), x, a.empty_weight(), n, keep)  # loads the kernels before the capture
    torch.cuda.synchronize()
    pool = torch.cuda.graph_pool_handle()
    gb, gd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gb, pool=pool):
        ob, lb = _step(b, x, wb, n, keep)
    with torch.cuda.graph(gd, pool=pool):
        od, ld = _step(d, x, wd, n, keep)
    for t in range(3):
        x["qkv"].copy_(rows(71 + t, 1, n, 4 + 2 * g, hd))
        oa, la = _step(a, x, wa, n, keep)
        gb.replay()
        torch.cuda.synchronize()
        ob_, lb_ = ob.clone(), lb.clone()
        gd.replay()
        torch.cuda.synchronize()
        for got in ((ob_, lb_, wb, b), (od, ld, wd, d)):
            assert torch.equal(got[0], oa) and torch.equal(got[1], la) and torch.equal(got[2], wa)
            assert torch.equal(got[3].lens, a.lens) and torch.equal(got[3].k.view(torch.uint8), a.k.view(torch.uint8))
    assert_device_ok()


@pytest.mark.parametrize("n", [1, 150])
def test_calls_on_other_streams_at_once(n):
    """Two caches, each on its own stream, and the explicit stream argument."""
    lens = [3000]
    cs = [filled(1, 3000, 2, 128, 64, lens, seed=80 + i) for i in range(2)]
    qs = [queries(90 + i, 1, n, 8, 128) for i in range(2)]
    want = [c.attend(q) for c, q in zip(cs, qs)]
    wwant = []
    for c, q, (_, lse) in zip(cs, qs, want):
        wwant.append(c.weigh(q, lse, c.empty_weight()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(4):
        got, wgot = [], []
        for c, q, s in zip(cs, qs, streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append(c.attend(q, stream=s))
            w = c.empty_weight()
            s.wait_stream(torch.cuda.current_stream())
            wgot.append(c.weigh(q, got[-1][1], w, stream=s))
        torch.cuda.synchronize()
        for (o, lse), (ro, rl), w, rw in zip(got, want, wgot, wwant):
            assert torch.equal(o, ro) and torch.equal(lse, rl) and torch.equal(w, rw)


def test_results_do_not_depend_on_the_batch_or_the_run():
    lens = [700, 700, 700]
    c = filled(3, 700, 2, 128, 64, lens, seed=100)
    q = queries(101, 3, 1, 8, 128)
    a, _ = c.attend(q)
    b, _ = c.attend(q)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ corners

def scattered(batch, cap, g, hd, block, lens, seed):
    """A cache of random bytes and scales (powers of two)."""
    c = A.KVCache8.empty(batch, cap, g, hd, block)
    gen = torch.Generator("cuda").manual_seed(seed)
    for t in (c.k, c.v):
        u = t.view(torch.uint8)
        u.copy_(torch.randint(0, 0x70, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
        u.bitwise_or_(torch.randint(0, 2, t.shape, generator=gen, device="cuda", dtype=torch.uint8) << 7)
    for t in (c.k_scale, c.v_scale):
        t.copy_(2.0 ** torch.randint(-9, -6, t.shape, generator=gen, device="cuda").float())
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return c


@pytest.mark.parametrize("lens,n,g,group,hd,block,causal", [
    ([9000], 1, 200, 1, 64, 16, False),              # more blocks in a key range than scales kept beside it
    ([50 + i for i in range(70)], 40, 1, 1, 64, 16, True),  # more sequences than lengths kept beside the items
    ([200, 90], 2, 1, 136, 64, 32, False),           # more heads on a key head than a query tile has rows
    ([200, 0, 90], 1, 2, 40, 128, 16, True),
    ([40_000], 3, 1, 1, 128, 64, False),
    ([2600], 34, 1, 4, 128, 128, True),              # one pair of query tiles, its keys split many ways
    ([1], 300, 1, 2, 64, 16, True),                  # one key: all rows but the last see nothing
])
def test_corner_sizes(lens, n, g, group, hd, block, causal):
    c = scattered(len(lens), max(lens) + 9, g, hd, block, lens, seed=110)
    q = queries(111, len(lens), n, g * group, hd) * 0.2
    _, lse = check_attend(c, q, lens, causal)
    check_weigh(c, q, lse, lens, causal)


@pytest.mark.parametrize("n", [1, 60])
def test_an_output_of_odd_sixteen_byte_rows(n):
    """Rows of o that start 16, not 32, bytes from a 32-byte boundary."""
    c = scattered(1, 300, 2, 64, 16, [300], seed=112)
    q = queries(113, 1, n, 4, 64)
    want, _ = c.attend(q)
    raw = torch.zeros((n * (4 * 64 + 8) + 8,), dtype=torch.bfloat16, device="cuda")
    out = raw[8:].as_strided((1, n, 4, 64), (n * 264, 264, 64, 1))
    c.attend(q, out=out)
    assert torch.equal(out, want)


def test_no_queries_still_decay_the_weights():
    c = scattered(2, 100, 2, 64, 16, [100, 33], seed=114)
    w = torch.ones((2, 2, c.n_blocks), device="cuda")
    q = torch.zeros((16,), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((4,), device="cuda")
    desc = L.Kv8Query(0, 0, 0, 2, 0, 0, 0, 0.0, 0)
    L.cosmot_kv8_weigh(c.desc, desc, q.data_ptr(), 128, lse.data_ptr(), 0.25, w.data_ptr(),
                       torch.cuda.current_stream().cuda_stream)
    live = torch.arange(c.n_blocks, device="cuda") * 16 < c.lens[:, None]
    assert torch.equal(w, torch.where(live[:, None], 0.25, 1.0).expand_as(w))
    assert_device_ok()


@pytest.mark.parametrize("n", [1, 150])
def test_outputs_made_here_wait_for_the_current_stream(n):
    """A call on another stream takes its outputs from the current stream's memory,
    which may still be in use there."""
    c = scattered(1, 2000, 2, 64, 64, [2000], seed=115)
    q = queries(116, 1, n, 4, 64)
    want, wl = c.attend(q)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.ones((1 << 26,), device="cuda")
    for _ in range(5):
        busy = torch.empty_like(want)
        for _ in range(20):
            big.mul_(1.0)
        busy.fill_(3.0)  # behind the work above, in memory that is free (to this stream) after the next line
        del busy
        o, lse = c.attend(q, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("n", [1, 40, 150])
def test_the_debug_build_gives_the_same_and_finds_nothing(n):
    """Every store index is checked there."""
    D, R = L.lib_debug(), L.lib()
    outs = []
    for lib in (R, D):
        L._lib = lib
        try:
            c = filled(2, 700, 2, 64, 16, [333, 77], seed=117)
            w = c.empty_weight()
            o, lse = _step(c, {"qkv": rows(118, 2, n, 8, 64)}, w, n, 9)
            torch.cuda.synchronize()
            assert_device_ok()
        finally:
            L._lib = R
        outs.append((o, lse, w, c.lens, c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale.nan_to_num()))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_the_python_layer_refuses_what_does_not_fit():
    c = scattered(2, 100, 2, 64, 16, [100, 33], seed=120)
    q = queries(121, 2, 3, 4, 64)
    o, lse = c.attend(q)
    w = c.empty_weight()
    for call in (lambda: c.attend(q.float()), lambda: c.attend(q.cpu()), lambda: c.attend(q[:1]), lambda: c.attend(q[0]),
                 lambda: c.attend(q, out=o[:, :2]), lambda: c.attend(q, out=o.float()), lambda: c.attend(q, lse=lse[:, :, :2]),
                 lambda: c.attend(q, lse=lse.transpose(1, 2)), lambda: c.weigh(q, lse[:1], w), lambda: c.weigh(q, lse, w[:, :1]),
                 lambda: c.weigh(q, lse, w.double()), lambda: c.weigh(q[:, :0], lse[:, :, :0], w), lambda: c.weigh(q, lse.cpu(), w),
                 lambda: c.evict(w[:, :, 1:], 2), lambda: c.evict(w.cpu(), 2), lambda: c.store(q, q),
                 lambda: c.store(q[:, :, :2], q[:, :2, :2]), lambda: c.store(q[:, :, :2].float(), q[:, :, :2].float()),
                 lambda: c.evict(w, 2, workspace=torch.empty((8,), dtype=torch.uint8, device="cuda")),
                 lambda: A.KVCache8(c.k, c.v[:, :50], c.k_scale, c.v_scale, c.lens, 16),
                 lambda: A.KVCache8(c.k, c.v, c.k_scale, c.v_scale, c.lens, 24),
                 lambda: A.KVCache8(c.k, c.v, c.k_scale[:, :, 1:], c.v_scale, c.lens, 16),
                 lambda: A.KVCache8(c.k, c.v, c.k_scale, c.v_scale, c.lens.long(), 16)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.attend(queries(121, 2, 3, 3, 64)), lambda: c.attend(q, n_new=101), lambda: c.attend(q, n_new=-1),
                 lambda: c.attend(q, max_len=-1), lambda: c.attend(q, softmax_scale=-1.0), lambda: c.weigh(q, lse, w, decay=-1.0),
                 lambda: c.evict(w, 0), lambda: c.evict(w, 2, first_rows=-1), lambda: c.store(*[rows(1, 2, 101, 2, 64)] * 2)):
        with pytest.raises(L.CosmotError):
            call()
    empty, none = c.attend(q[:, :0])
    assert empty.shape == (2, 0, 4, 64) and none.shape == (2, 4, 0)
    c.store(q[:, :0, :2], q[:, :0, :2])
    assert torch.equal(c.attend(q)[0], o)
    assert_device_ok()

"""The 8-bit cache at sizes whose work plans the small ones do not reach: whole items beside split ones, CTAs that
weigh several key ranges (alone and in clusters), long causal prompts, the radix selection; a batch against its
sequences; and a layer's own rows."""

import math

import pytest
import torch

import kv8_plain as P
from gpu_helpers import assert_device_ok

pytestmark = pytest.mark.gpu

from flow_matching_dit_cosmot_b200 import _lib as L  # noqa: E402
from flow_matching_dit_cosmot_b200 import api as A  # noqa: E402
from test_gpu_kv8 import check_attend, check_weigh, dequant, filled, queries, rows, scattered  # noqa: E402


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def split_plan(items, n_kt):
    """(whole items, items of k ranges, items of k + 1 ranges, k) as the tile attention plans them: the items of the last
    wave are split into m full waves, m (longest range + 4 tiles) + ranges / 48 + 2 the least."""
    tail, best, plan = items % sms(), n_kt + 4.0, (items, 0, 0, 1)
    for m in range(1, 7 if tail else 1):
        k, hi = m * sms() // tail, m * sms() % tail
        cut = min(k, 255, n_kt // 2 if 2 * min(k, 255) > n_kt else k)
        if cut != k or 2 * (cut + 1) > n_kt:
            hi = 0
        k = cut
        if k < 1 or (k == 1 and hi < tail):
            continue
        cost = -(-n_kt // k) + (m - 1) * -(-n_kt // (k + 1 if hi else k)) + 4.0 * m + (tail * k + hi) / 48 + 2
        if cost < best:
            best, plan = cost, (items - tail, tail - hi, hi, k)
    return plan


BIG = [  # lengths, n_q, kv heads, group, head_dim, block, causal: what attend plans, and the items of weigh
    ([3000, 2700], 1300, 16, 1, 64, 64, False),
    ([3000, 1303], 1300, 16, 1, 128, 16, True),      # a causal prompt behind a history
    ([2900, 0, 900], 650, 9, 2, 64, 128, True),      # a prompt of which a sequence has nothing, another a part
    ([4100], 2000, 20, 1, 128, 32, False),
]


@pytest.mark.parametrize("lens,n,g,group,hd,block,causal", BIG)
def test_whole_and_split_items_and_many_key_ranges_a_cta(lens, n, g, group, hd, block, causal):
    cap = max(lens) + 3
    whole, lo, hi, k = split_plan(len(lens) * g * -(-n * group // 256), -(-cap // 128))
    assert whole >= sms() and k >= 1 and hi > 0 and lo + hi > 0, (whole, lo, hi, k)
    assert len(lens) * g * -(-cap // 256) > sms()
    c = scattered(len(lens), cap, g, hd, block, lens, seed=300)
    q = queries(301, len(lens), n, g * group, hd) * 0.2
    _, lse = check_attend(c, q, lens, causal)
    check_weigh(c, q, lse, lens, causal)


@pytest.mark.parametrize("n,group,block,causal", [(1100, 1, 64, False), (1030, 1, 128, True), (300, 4, 16, False), (700, 2, 32, True)])
def test_clusters_that_weigh_several_key_ranges(n, group, block, causal):
    """A bound on the lengths that is too small: clusters share the queries, and each takes more than one range."""
    lens = [9100, 4000]
    assert -(-n // (128 // group)) >= 8 and 2 * 2 * 4 * 2 <= sms() and 2 * 36 > sms() // 4  # four CTAs a cluster, two ranges each
    c = scattered(2, 9216, 1, 128, block, lens, seed=310)
    q = queries(311, 2, n, group, 128) * 0.2
    _, lse = c.attend(q, causal=causal)
    K, _ = dequant(c, lens)
    w = torch.rand((2, 1, c.n_blocks), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    ref, bound = P.weigh(q, K, lse, lens, block, causal, w, 0.5)
    one = w.clone()
    c.weigh(q, lse, w, decay=0.5, causal=causal, max_len=300)
    c.weigh(q, lse, one, decay=0.5, causal=causal)
    torch.cuda.synchronize()
    assert_device_ok()
    for x in (w, one):
        assert bool(((x.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("n,lens", [(2048, [2048]), (3000, [3000, 3500])])
def test_long_causal_prompts(n, lens):
    c = filled(len(lens), max(lens), 2, 128, 64, lens, seed=320)
    q = queries(321, len(lens), n, 4, 128)
    _, lse = check_attend(c, q, lens, True)
    check_weigh(c, q, lse, lens, True)


def test_a_batch_gives_what_its_sequences_give_alone():
    """Split differently, so not bit for bit: both within the bound of one definition."""
    lens = [700, 3, 2100]
    for n in (1, 50, 200):
        c = filled(3, 2100, 2, 128, 64, lens, seed=330)
        q = queries(331, 3, n, 8, 128)
        o, lse = check_attend(c, q, lens, False)
        for b, m in enumerate(lens):
            one = A.KVCache8(c.k[b:b + 1], c.v[b:b + 1], c.k_scale[b:b + 1], c.v_scale[b:b + 1], c.lens[b:b + 1], 64)
            check_attend(one, q[b:b + 1], [m], False)
            K, V = dequant(one, [m])
            _, _, bo, bl, _ = P.attend(q[b:b + 1], K, V, [m], False)
            ob, lb = one.attend(q[b:b + 1])
            assert bool(((ob[0].double() - o[b].double()).abs() <= 2 * bo[0]).all())
            assert bool(((lb[0].double() - lse[b].double()).abs() <= 2 * bl[0]).all())


# ------------------------------------------------------------------ the radix selection

def _bits(w):
    return w.view(torch.int32)


@pytest.mark.parametrize("kind", ["low bytes", "full", "special", "negative"])
@pytest.mark.parametrize("keep", [30, 517, 1100])
def test_evict_by_every_digit_of_the_weights(kind, keep):
    """More than 512 free blocks: the threshold is found digit by digit, the last ones too."""
    n_rows, block = 20_003, 16
    c = A.KVCache8.empty(2, n_rows, 2, 64, block)
    gen = torch.Generator("cuda").manual_seed(340)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 120, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
    lens = [n_rows, 15_000]
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    shape = (2, 2, c.n_blocks)
    if kind == "low bytes":  # equal but for the last two digits
        w = (torch.randint(0, 1 << 10, shape, generator=gen, device="cuda", dtype=torch.int32) + 0x3f800000).view(torch.float32)
    else:
        w = torch.randn(shape, generator=gen, device="cuda") * torch.exp(3 * torch.randn(shape, generator=gen, device="cuda"))
        w = -w.abs() if kind == "negative" else (w.abs() if kind == "full" else w)
    if kind == "special":
        pick = torch.randint(0, 12, shape, generator=gen, device="cuda")
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, 2.0 ** -149, -2.0 ** -149)):
            w = torch.where(pick == i, torch.full_like(w, x), w)
        w.view(torch.int32)[pick == 7] = -1  # a NaN of the other sign
    w = w.contiguous()
    kb, vb, ks, vs = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu(), c.k_scale.cpu(), c.v_scale.cpu()
    wref, lref = P.evict(kb, vb, ks, vs, w.cpu(), lens, block, keep, 66, 300)
    c.evict(w, keep, 66, 300)
    torch.cuda.synchronize()
    assert_device_ok()
    assert c.lens.tolist() == lref
    assert torch.equal(_bits(w).cpu(), _bits(wref))
    assert torch.equal(c.k.view(torch.uint8).cpu(), kb) and torch.equal(c.v.view(torch.uint8).cpu(), vb)


# ------------------------------------------------------------------ a layer's rows

def test_a_layers_own_rows_go_through_the_cache():
    """The QKV rows of a layer (rotated by mRoPE), stored from their columns: text rows causally, then the DM rows over
    everything, as a streaming step does; the layer is finished on what the cache's attention gives."""
    import synth
    from flow_matching_dit_cosmot_b200.ulysses import UlyssesShard
    from gpu_helpers import to_dev
    from test_gpu_layer import LayerRun
    dims = synth.ModelDims(d_model=512, n_heads=4, n_kv_heads=2, head_dim=128, ffn=1024, rope_sections=(16, 24, 24))
    run = LayerRun(dims, synth.preset("droid").layout)
    n, n_ar = run.lay.n_tokens, run.lay.n_ar
    h = to_dev(run.h[0])
    before, out = h.clone(), torch.empty_like(h)
    sh = UlyssesShard(run.layer, run.seq, 1, 0)
    sh.pre(h)
    qkv = sh.qkv_local.view(1, n, 8, 128)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    c = A.KVCache8.empty(1, n, 2, 128, 32)
    c.store(k[:, :n_ar], v[:, :n_ar])
    o_ar, _ = check_attend(c, q[:, :n_ar], [0], True, n_new=n_ar)
    c.advance(n_ar)
    c.store(k[:, n_ar:], v[:, n_ar:])
    o_dm, _ = check_attend(c, q[:, n_ar:], [n_ar], False, n_new=n - n_ar)
    # the cached rows are the layer's, rounded to e4m3: half a step of 2^-4 of each element above the scale's smallest
    # normal (2^-6), 2^-10 scales below
    for got, want in zip(dequant(c, [n]), (k, v)):
        scale = (c.k_scale if want is k else c.v_scale).double().repeat_interleave(32, 2)[:, :, :n].transpose(1, 2)[..., None]
        assert bool(((got - want.double()).abs() <= torch.maximum(want.double().abs() * 2.0 ** -4, scale * 2.0 ** -10)).all())
    sh.recv2[0].copy_(torch.cat([o_ar, o_dm], 1).view(n, 512))
    sh.post(h, out, 0.8, 0.7)
    torch.cuda.synchronize()
    assert_device_ok()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(h).all())
    noisy = n - run.lay.n_noisy
    assert torch.equal(h[:noisy], before[:noisy]) and not torch.equal(h[noisy:], before[noisy:])

"""What the 8-bit cache's calls promise around their numbers: failures of others,
lengths outside the cache, streams, descriptors, and the work plans of large calls."""

import math

import pytest
import torch

import kv8_plain as P
from gpu_helpers import assert_device_ok

pytestmark = pytest.mark.gpu

from flow_matching_dit_cosmot_b200 import _lib as L  # noqa: E402
from flow_matching_dit_cosmot_b200 import api as A  # noqa: E402
from test_gpu_kv8 import check_attend, check_weigh, dequant, filled, queries, rows, scattered  # noqa: E402,F401


def test_calls_after_a_failure_end_and_the_next_ones_are_right():
    """A status word that holds a failure ends every wait at once; what is in flight is waited for all the same."""
    lens = [703, 650]
    c = filled(2, 710, 2, 128, 64, lens, seed=201)
    q = queries(202, 2, 260, 8, 128)
    want, wl = c.attend(q)
    w = c.weigh(q, wl, c.empty_weight())
    assert_device_ok()
    L.cosmot_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        o, lse = c.attend(q)
        c.weigh(q, lse, c.empty_weight())
    torch.cuda.synchronize()
    st = L.cosmot_get_device_status(torch.cuda.current_stream().cuda_stream)
    assert st == (L.COSMOT_ERR_TIMEOUT, L.COSMOT_SITE_SELFTEST)
    o, lse = c.attend(q)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert torch.equal(c.weigh(q, lse, c.empty_weight()), w)
    assert_device_ok()


# ------------------------------------------------------------------ a length outside the cache

def _status():
    return L.cosmot_get_device_status(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("n", [1, 40, 150, 260])
@pytest.mark.parametrize("bad,nearest", [(-3, 0), (401, 400), (2 ** 31 - 1, 400), (-2 ** 31, 0)])
def test_a_bad_length_costs_no_other_sequence_its_results(n, bad, nearest):
    """The sequence takes the nearest length inside; the others' outputs, weights and blocks are the good batch's."""
    lens = [nearest, 333, 400]
    good = scattered(3, 400, 2, 128, 32, lens, seed=210)
    c = scattered(3, 400, 2, 128, 32, [bad, 333, 400], seed=210)
    q = queries(211, 3, n, 8, 128) * 0.2
    want, wl = good.attend(q)
    ww = good.weigh(q, wl, good.empty_weight())
    assert_device_ok()
    o, lse = c.attend(q)
    w = c.weigh(q, lse, c.empty_weight())
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(w, ww)
    good.evict(ww, 5)
    c.evict(w, 5)
    torch.cuda.synchronize()
    assert torch.equal(w, ww) and torch.equal(c.lens, good.lens)
    assert torch.equal(c.k.view(torch.uint8), good.k.view(torch.uint8))
    assert _status() == (L.COSMOT_ERR_BOUNDS, 400)
    assert_device_ok()


def test_a_store_without_room_costs_other_calls_nothing():
    """The report stays unread while the layer's products and bf16 attention and this cache's own calls run."""
    from test_gpu_layer import MEDIUM, LayerRun
    import synth
    from gpu_helpers import to_dev
    run = LayerRun(MEDIUM, synth.preset("droid").layout)
    first, again = to_dev(run.h), to_dev(run.h)
    out, out2 = torch.empty_like(first), torch.empty_like(first)
    run.layer.forward(first, out, 0.8, 0.7, run.seq)
    assert_device_ok()
    c = scattered(2, 300, 2, 64, 16, [296, 100], seed=212)
    before = c.k.view(torch.uint8).clone()
    x = rows(214, 2, 8, 2, 64)
    c.store(x, x)  # sequence 0 has no room for 8 rows
    run.layer.forward(again, out2, 0.8, 0.7, run.seq)
    c.lens.copy_(torch.tensor([296, 108], dtype=torch.int32))
    q = queries(213, 2, 200, 4, 64) * 0.2
    o, lse = c.attend(q)
    torch.cuda.synchronize()
    assert torch.equal(again, first) and torch.equal(out2, out)
    assert torch.equal(c.k.view(torch.uint8)[0], before[0])
    assert _status() == (L.COSMOT_ERR_BOUNDS, 400)
    o2, lse2 = check_attend(c, q, [296, 108], False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_failure_is_read_before_a_report_and_neither_is_lost():
    c = scattered(1, 64, 1, 64, 16, [64], seed=220)
    x = rows(221, 1, 1, 1, 64)
    c.store(x, x)
    L.cosmot_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream)
    assert _status() == (L.COSMOT_ERR_TIMEOUT, L.COSMOT_SITE_SELFTEST)
    assert _status() == (L.COSMOT_ERR_BOUNDS, 400)
    assert_device_ok()


# ------------------------------------------------------------------ rows apart, value scales far apart

@pytest.mark.parametrize("n", [3, 8, 60, 300])
def test_a_row_does_not_depend_on_the_rows_beside_it(n):
    """Keys that grow along the cache: a row's maximum moves many times, at its own keys whatever the others do."""
    c = scattered(1, 1300, 1, 64, 16, [1300], seed=240)
    c.k_scale.copy_(2.0 ** torch.linspace(-12, -3, c.n_blocks, device="cuda").floor())
    q = queries(241, 1, n, 2, 64)
    q[:, ::2] *= 0.25
    o, lse = c.attend(q)
    alone = q.clone()
    alone[:, 1::2] = 0
    oa, la = c.attend(alone)
    assert torch.equal(o[:, ::2], oa[:, ::2]) and torch.equal(lse[:, :, ::2], la[:, :, ::2])
    check_attend(c, q, [1300], False)


@pytest.mark.parametrize("n,block,large,small", [
    *((n, 32, a, b) for n in (1, 3, 8) for a, b in ((20, -13), (40, -40), (3, -25), (-13, 20))),
    *((n, 128, a, b) for n in (1, 40, 150, 300) for a, b in ((20, -13), (40, -40), (3, -25), (-13, 20))),
    *((n, block, a, b) for n in (40, 150, 300) for block in (16, 32, 64) for a, b in ((10, -10), (-30, -38), (40, 20), (-12, 8)))])
@pytest.mark.parametrize("causal", [False, True])
def test_a_large_scale_over_small_bytes_hides_no_other_value(n, block, large, small, causal):
    """The bound is relative to the values, not to their blocks' scales: a block of a large scale whose rows are zero
    (an outlier row that went, or that the mask hides) leaves the others' digits alone.  More than 32 packed rows: the
    blocks of an aligned run of 128 rows have scales within 2^22."""
    lens = [1300, 530]
    nb = -(-1300 // block)
    c = filled(2, 1300, 2, 128, block, lens, seed=230)
    c.v_scale[:] = 2.0 ** small * torch.tensor([1.0, 2.0, 4.0], device="cuda").repeat(nb)[:nb]
    for h, first, step in ((0, 1, 4), (1, 0, 3)):
        c.v_scale[:, h, first::step] = 2.0 ** large
        for j in range(first, nb, step):
            c.v.view(torch.uint8)[:, block * j:block * (j + 1), h] = 0
    for b, m in enumerate(lens):  # nothing reads the scales of blocks without a row
        c.v_scale[b, :, -(-m // block):] = math.nan
    q = queries(231, 2, n, 4, 128)
    check_attend(c, q, lens, causal)


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("large,small", [(20, -13), (22, -14)])
def test_scales_too_far_apart_in_one_run_lose_the_digits_that_are_stated(n, large, small):
    """Blocks of 32 in runs of 128 rows, scales 2^(22 + d) apart: weights are right to 2^(d - 33) of the largest."""
    lens, block, d = [1300], 32, large - small - 22
    c = filled(1, 1300, 1, 128, block, lens, seed=232)
    c.v_scale[:] = 2.0 ** small
    c.v_scale[:, :, 1::4] = 2.0 ** large
    for j in range(1, c.n_blocks, 4):
        c.v.view(torch.uint8)[:, block * j:block * (j + 1)] = 0
    q = queries(233, 1, n, 2, 128)
    o, lse = c.attend(q)
    K, V = dequant(c, lens)
    ro, rl, bo, bl, _ = P.attend(q, K, V, lens, False)
    for h in range(2):
        w = torch.exp(q[0, :, h].double() @ K[0, :, 0].T / math.sqrt(128) - rl[0, h][:, None])
        bo[0, :, h] += 2.0 ** (d - 33) * w.amax(1, keepdim=True) * V[0, :, 0].abs().sum(0)
    assert bool(((o.double() - ro).abs() <= bo).all()) and bool(((lse.double() - rl).abs() <= bl).all())
    assert_device_ok()


# ------------------------------------------------------------------ the debug build

@pytest.mark.parametrize("lens,n,g,group,block,keep", [([5000], 1, 2, 4, 16, 40), ([3000, 700], 40, 2, 1, 64, 7),
                                                       ([2600, 0, 90], 200, 1, 2, 128, 5), ([12_000], 3, 1, 8, 32, 600)])
def test_the_debug_build_agrees_on_split_keys_and_moves(lens, n, g, group, block, keep):
    """Its checks of the partial results' places and of the moves' sources and destinations find nothing."""
    outs = []
    release = L.lib()
    for lib in (release, L.lib_debug()):
        L._lib = lib
        try:
            c = scattered(len(lens), max(lens), g, 64, block, lens, seed=250)
            q = queries(251, len(lens), n, g * group, 64) * 0.2
            o, lse = c.attend(q)
            w = c.weigh(q, lse, c.empty_weight())
            c.evict(w, keep, 20, 30)
            torch.cuda.synchronize()
            assert_device_ok()
        finally:
            L._lib = release
        outs.append((o, lse, w, c.lens, c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ streams

def _late(t, seconds=0.02):
    """A copy of t that the current stream makes only after some work."""
    out = torch.zeros_like(t)
    torch.cuda._sleep(int(seconds * 1.5e9))
    out.copy_(t)
    return out


@pytest.mark.parametrize("n", [1, 150])
def test_a_streaming_step_on_another_stream_is_the_same(n):
    """The documented step with stream= on every call, its inputs still being made on the current stream."""
    make = lambda: scattered(2, 900, 2, 64, 16, [300, 41], seed=260)  # noqa: E731
    a, b = make(), make()
    wa, wb = a.empty_weight(), b.empty_weight()
    s = torch.cuda.Stream()
    for t in range(3):
        x = rows(261 + t, 2, n, 8, 64) * 0.2
        a.store(x[:, :, 4:6], x[:, :, 6:])
        oa, la = a.attend(x[:, :, :4], n_new=n)
        a.weigh(x[:, :, :4], la, wa, n_new=n)
        a.advance(n)
        a.evict(wa, 12, first_rows=10, last_rows=n)
        torch.cuda.synchronize()
        y = _late(x)
        b.store(y[:, :, 4:6], y[:, :, 6:], stream=s)
        ob, lb = b.attend(y[:, :, :4], n_new=n, stream=s)
        b.weigh(y[:, :, :4], lb, wb, n_new=n, stream=s)
        b.advance(n, stream=s)
        b.evict(wb, 12, first_rows=10, last_rows=n, stream=s)
        torch.cuda.synchronize()
        for p, q in ((oa, ob), (la, lb), (wa, wb), (a.lens, b.lens), (a.k.view(torch.uint8), b.k.view(torch.uint8)),
                     (a.v_scale, b.v_scale)):
            assert torch.equal(p, q)
    assert_device_ok()


def test_store_on_another_stream_waits_for_its_inputs():
    a, b = (scattered(1, 200, 2, 64, 16, [30], seed=265) for _ in range(2))
    x = rows(266, 1, 100, 4, 64)
    a.store(x[:, :, :2], x[:, :, 2:])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = _late(x)
    b.store(y[:, :, :2], y[:, :, 2:], stream=s)
    b.advance(100, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and b.lens.tolist() == [130]


def test_weigh_on_another_stream_waits_for_its_inputs():
    c = scattered(1, 900, 2, 64, 16, [900], seed=267)
    q = queries(268, 1, 3, 4, 64) * 0.2
    _, lse = c.attend(q)
    want = c.weigh(q, lse, c.empty_weight())
    torch.cuda.synchronize()
    w = _late(c.empty_weight() + 1) - 1
    c.weigh(q, lse, w, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(w, want)


# ------------------------------------------------------------------ the cache object

def test_replacing_a_tensor_is_refused_and_copying_the_new_lengths_works():
    """Out-of-place eviction returns new lengths; assigned, they would be without effect."""
    a, b = (scattered(1, 300, 2, 64, 16, [300], seed=270) for _ in range(2))
    w = torch.rand((1, 2, a.n_blocks), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    wa, lens = a.evict(w, 7, in_place=False)
    with pytest.raises(AttributeError):
        a.lens = lens
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(a, name, getattr(b, name))
    a.lens.copy_(lens)
    a.lens += 1
    a.lens -= 1
    wb = w.clone()
    b.evict(wb, 7)
    q = queries(271, 1, 40, 4, 64) * 0.2
    assert torch.equal(a.lens, b.lens) and torch.equal(wa, wb)
    assert torch.equal(a.attend(q)[0], b.attend(q)[0])


# ------------------------------------------------------------------ short caches

@pytest.mark.parametrize("n", [1, 7, 30, 300])
@pytest.mark.parametrize("group", [1, 8])
def test_lse_of_a_few_keys_keeps_its_digits(n, group):
    """Sums near one, logarithms near zero: what the weights are kept times must not cost lse its last digits."""
    for seed in range(6):
        lens = [1, 2, 3, 1, 5, 2]
        c = scattered(6, 5, 8, 64, 64, lens, seed=280 + seed)
        for scale in (0.2, 0.02):
            q = (queries(290 + seed, 6, n, 8 * group, 64) * scale).to(torch.bfloat16)
            check_attend(c, q, lens, False)
            check_attend(c, q, lens, True)


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("exponent", [-31, 25])
def test_lse_does_not_depend_on_the_size_of_the_values(n, exponent):
    lens = [1, 2, 17, 91]
    for seed in range(4):
        c = scattered(4, 100, 8, 64, 16, lens, seed=300 + seed)
        q = (queries(310 + seed, 4, n, 16, 64) * 0.2).to(torch.bfloat16)
        _, lse = check_attend(c, q, lens, False)
        c.v_scale.mul_(2.0 ** exponent)
        _, far = check_attend(c, q, lens, False)
        assert torch.equal(lse, far)

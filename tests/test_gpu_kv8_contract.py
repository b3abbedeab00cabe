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

"""The 8-bit cache's largest sizes on the host (no GPU): what does not fit is refused before anything is counted in 32 bits."""

import ctypes

import pytest

from flow_matching_dit_cosmot_b200 import _lib as L
from test_kv8 import cache, query


@pytest.mark.parametrize("n_kv,n_q", [(60_000, 2 ** 30 - 1), (60_000, 200_000), (4, 2 ** 62), (4, 2 ** 63 - 1), (30_000, 2 ** 29)])
def test_more_work_items_than_a_grid_counts_are_refused_by_the_workspace_too(n_kv, n_q):
    lib = L.lib()
    c = cache(batch=1, n_kv_heads=n_kv, ld=n_kv * 128)
    q = query(n_q=n_q, q_batch_stride=n_q, o_batch_stride=n_q, n_heads=n_kv)
    n = ctypes.c_size_t(0)
    assert lib.cosmot_kv8_attention_workspace(ctypes.byref(c), ctypes.byref(q), ctypes.byref(n)) == L.COSMOT_ERR_UNSUPPORTED
    assert lib.cosmot_kv8_attention(ctypes.byref(c), ctypes.byref(q), 256, n_kv * 128, 256, n_kv * 128, None, 256, 1 << 60,
                                    None) == L.COSMOT_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_kv,n_q", [(1, 2 ** 30 - 1), (32, 1_000_000), (65_535, 33)])
def test_the_largest_calls_that_fit_have_a_workspace_of_a_wave_at_most(n_kv, n_q):
    """Only items of the last wave are split, into six waves of ranges at most."""
    c = cache(batch=1, n_kv_heads=n_kv, ld=n_kv * 128, capacity=1_000_000)
    need = L.cosmot_kv8_attention_workspace(c, query(n_q=n_q, q_batch_stride=n_q, o_batch_stride=n_q, n_heads=n_kv))
    assert 0 <= need <= 6 * 160 * 256 * (128 * 4 + 8) + 256


@pytest.mark.parametrize("n_q,group,want", [(2 ** 25 + 1, 1, L.COSMOT_ERR_UNSUPPORTED), (2 ** 22 + 1, 8, L.COSMOT_ERR_UNSUPPORTED),
                                            (2 ** 30 - 1, 1, L.COSMOT_ERR_UNSUPPORTED)])
def test_weighing_more_rows_than_its_waits_allow_is_refused(n_q, group, want):
    c = cache(batch=1)
    q = query(n_q=n_q, q_batch_stride=n_q, o_batch_stride=n_q, n_heads=2 * group)
    assert L.lib().cosmot_kv8_weigh(ctypes.byref(c), ctypes.byref(q), 256, 2 * group * 128, 256, 1.0, 256, None) == want

"""Pins of the NumPy reference of the key-value cache (CPU) where the GPU tests rely on more than finite values."""
import numpy as np

from oracle import kv_cache as ref


def test_reference_eviction_around_a_bad_page_by_hand():
    """Six slots on three pages, the second of them none of the pool's: its slots before the budget stay."""
    rng = np.random.default_rng(2)
    c = ref.Cache(rng, [6], 1, 64, 2, "bf16")
    p, _, s = c.at(0, np.arange(6))
    c.weight[p, 0, s] = [0.5, 0.1, 9.0, 9.0, 0.3, 0.9]
    c.position[p, 0, s] = [0, 1, 2, 3, 4, 5]
    rows = c.rows(0, np.arange(6))[0][0].copy()
    c.table[0, 1] = -1
    # Budget 3: slot 2 takes up a place, and of the rest 5 (0.9) and 0 (0.5) are best: 5 goes to slot 1.
    assert list(c.evict(3, 0)) == [3]
    np.testing.assert_array_equal(c.rows(0, [0, 1])[0][0], rows[[0, 5]])
    assert list(c.weight[p[:2], 0, s[:2]]) == [np.float32(0.5), np.float32(0.9)]
    np.testing.assert_array_equal(c.weight[p[2:4], 0, s[2:4]], [9.0, 9.0])   # the page taken out is as it was
    # Budget 5: both slots of that page count; the three best of the other four.
    c.weight[p, 0, s] = [0.5, 0.1, 9.0, 9.0, 0.3, 0.9]
    before = c.rows(0, [0, 1, 4, 5])[0][0].copy()
    assert list(c.evict(5, 0)) == [5]
    np.testing.assert_array_equal(c.rows(0, [0, 1, 4])[0][0], before[[0, 3, 2]])

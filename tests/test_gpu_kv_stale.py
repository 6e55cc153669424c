"""Reservations for rows whose entries name pages that nobody holds (a table that
began as zeros, a row whose pages were given back elsewhere), against the oracle."""

import numpy as np
import pytest

from gpu_util import announce
from test_gpu_kv_pages import full_cache, run_reserve

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,P,H", [(64, 16, 2), (128, 64, 3)])
@pytest.mark.parametrize("B", [1, 9, 1500])
def test_a_table_of_zeros(D, P, H, B):
    """Every entry names page 0, which is free: one row gets it, no count falls below 0."""
    announce(f"kv reserve over zeros D={D} B={B}")
    rng = np.random.default_rng(B)
    cache, ref = full_cache(rng, 2 * B + 3, H, D, P)
    lens = rng.integers(0, 2 * P, B)
    lens[0] = 5
    table, refs = np.zeros((B, 3), np.int32), np.zeros(2 * B + 3, np.int32)
    run_reserve(cache, ref, table, lens, refs, 4, D, P)
    assert refs.min() == 0 and refs.max() == 1 and refs.sum() == sum((n + 3) // P - n // P + 1 for n in lens)


def test_entries_that_name_each_others_new_pages():
    """Free pages in the order that others get them, beside shared ones and some that are held alone."""
    announce("kv reserve, entries that are free")
    rng = np.random.default_rng(1)
    P, D, H, B, pages = 16, 64, 2, 400, 1000
    cache, ref = full_cache(rng, pages, H, D, P)
    refs = np.zeros(pages, np.int32)
    table = np.full((B, 2), -1, np.int32)
    table[:, 0] = rng.permutation(B)  # pages 0 .. 399: free, and the first that are given out
    for b in range(0, B, 5):  # rows b and b + 1 share a page, row b + 2 has its own
        table[b:b + 2, 0], table[b + 2, 0] = 600 + b, 601 + b
        refs[600 + b], refs[601 + b] = 2, 1
    refs[3] = -2  # given back once too often
    lens = rng.integers(1, P, B)
    run_reserve(cache, ref, table, lens, refs, 9, D, P)
    assert refs.min() >= 0

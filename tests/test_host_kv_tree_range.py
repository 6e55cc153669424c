"""CPU check of the tree attention's running maximum and sum (the step that the
kernel and the dry run share), against softmax's in 64 bits."""

import ctypes

import numpy as np
import pytest

from test_host_dryrun import dl  # noqa: F401  (the dry-run library)


def row(dl, scores, step):  # noqa: F811
    s = np.ascontiguousarray(scores, dtype=np.float32)
    m, l = ctypes.c_float(), ctypes.c_float()
    dl.brq_dryrun_tree_row.restype = None
    dl.brq_dryrun_tree_row(ctypes.c_void_p(s.ctypes.data), len(s), step, ctypes.byref(m), ctypes.byref(l))
    return m.value, l.value


@pytest.mark.parametrize("at", [0.0, -127.0, -129.0, -200.0, -1500.0, -3e4, 129.0, 200.0, 3e4])
@pytest.mark.parametrize("n,step,first", [(1, 32, 0), (32, 32, 0), (33, 32, 32), (500, 32, 100), (500, 4, 7), (64, 32, 63)])
def test_running_maximum_of_scores_far_from_zero(dl, at, n, step, first):  # noqa: F811
    """Scores around `at`, the first ones masked."""
    rng = np.random.default_rng(n + step)
    s = np.float32(at + 3 * rng.standard_normal(n))
    s[:first] = -np.inf
    m, l = row(dl, s, step)
    x = s.astype(np.float64)
    # a difference of scores is off by the rounding of either side, 2^-23 of the
    # largest in all, an addition by 2^-24; the maximum may be summed up in as many steps
    tol = 2.0 ** -22 * (np.abs(x[first:]).max() + n)
    assert np.isfinite(l) and l >= 0.5
    assert abs((m + np.log2(l)) - (x.max() + np.log2(np.exp2(x - x.max()).sum()))) <= tol * 1.5


@pytest.mark.parametrize("low", [-200.0, -130.0, -3e4])
def test_low_scores_before_ordinary_ones(dl, low):  # noqa: F811
    """What a row saw first does not matter next to a score 100 above it."""
    s = np.full(96, low, np.float32)
    s[64:] = 1.0
    assert row(dl, s, 32) == (1.0, 32.0)
    assert row(dl, s[::-1], 32) == (1.0, 32.0)


def test_a_row_that_sees_nothing(dl):  # noqa: F811
    assert row(dl, np.full(70, -np.inf), 32) == (-np.inf, 0.0)
    assert row(dl, [], 32) == (-np.inf, 0.0)

"""CPU check of the polynomial that gelu's epilogue uses, with its coefficients, in 64 bits."""

import ctypes

import numpy as np

from test_host_dryrun import dl  # noqa: F401  (dl: the dry-run library)


def tail(dl, z):  # noqa: F811
    f = dl.brq_dryrun_gelu_tail
    f.argtypes, f.restype = [ctypes.c_double], ctypes.c_double
    return np.array([f(x) for x in z])


def test_gelus_polynomial_is_as_near_as_it_says(dl):  # noqa: F811
    from scipy.special import erfcx
    z = np.concatenate((np.linspace(0, 12, 40001), np.geomspace(1e-9, 12, 2000)))
    off = np.abs(tail(dl, z) / erfcx(z) - 1)
    assert off.max() <= 1.4 * 2.0 ** -24
    # beyond, nothing is left of it in float32: the smallest number there is 2^-149
    z = np.linspace(12, 100, 1000)
    with np.errstate(under="ignore"):
        assert (np.abs(tail(dl, z)) * np.sqrt(2) * z * np.exp(-z ** 2) < 2.0 ** -150).all()

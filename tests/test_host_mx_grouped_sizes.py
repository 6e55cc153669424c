"""CPU check: grouped products of all sizes that the checks let through are launches that
can be made, of a kernel that there is."""

import itertools

import pytest

from test_host_dryrun import _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import B2, CODES, S2, SCALES, UNSUPPORTED, WS, Y

OFFS = 0x1300000000


def call(dl, T, E, m, n):  # noqa: F811
    nb = dl.brq_mx_grouped_matmul_workspace_bytes(T, E, m, n)
    return dl.brq_mx_grouped_matmul(CODES, SCALES, B2, S2, OFFS, T, E, m, n, None, Y, 1, m, WS if nb else None, nb, None)


@pytest.mark.parametrize("n", [32, 224, 256, 2048, 2080, 1 << 23, (1 << 23) + 32])
def test_sizes_up_to_a_launch(dl, n):  # noqa: F811
    taken = 0
    for T, E, m in itertools.product((1, 40000, (1 << 20) + 1, 260_000_000, 1 << 28),
                                     (1, 64, 700_000, 1 << 20), (1, 16, 17, 33, 1000, 1 << 20, 1 << 28)):
        if T * m > 1 << 33 or (T <= 1 << 20 and E > 64):  # (a walk through so many groups takes its time)
            continue
        dl.brq_dryrun_reset()
        st = call(dl, T, E, m, n)
        if st == UNSUPPORTED:
            units = -(-T // 16) + E  # at least as many as the kernel has
            assert units * -(-m // 32) >= 1 << 24
            assert dl.brq_mx_grouped_matmul_workspace_bytes(T, E, m, n) == 0
            continue
        _ok(dl, st, f"grouped {T}x{E}x{m}x{n}")
        taken += 1
    assert taken > 40


@pytest.mark.parametrize("n", [64, 512, 4096])
def test_every_mean(dl, n):  # noqa: F811
    """Rows a group from none to where tiles of either size take over."""
    for E, m in ((1, 64), (8, 4096), (100, 300)):
        for mean in (0, 1, 8, 9, 16, 17, 24, 25, 32, 33, 64, 65, 128, 200, 1000):
            dl.brq_dryrun_reset()
            _ok(dl, call(dl, max(1, mean * E), E, m, n), f"grouped {mean} rows of {E}")

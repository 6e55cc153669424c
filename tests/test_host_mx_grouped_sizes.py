"""CPU check: grouped products of all sizes that the checks let through are launches that
can be made, of a kernel that there is."""

import pytest

from test_host_dryrun import _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import B2, CODES, S2, SCALES, WS, Y

OFFS = 0x1300000000


def call(dl, T, E, m, n):  # noqa: F811
    nb = dl.brq_mx_grouped_matmul_workspace_bytes(T, E, m, n)
    return dl.brq_mx_grouped_matmul(CODES, SCALES, B2, S2, OFFS, T, E, m, n, None, Y, 1, m, WS if nb else None, nb, None)


@pytest.mark.parametrize("n", [64, 512, 4096])
def test_every_mean(dl, n):  # noqa: F811
    """Rows a group from none to where tiles of either size take over: units of 16 or 32 rows, or a tile's."""
    for E, m in ((1, 64), (8, 4096), (100, 300)):
        for mean in (0, 1, 8, 9, 16, 17, 24, 25, 32, 33, 64, 65, 128, 200, 1000):
            dl.brq_dryrun_reset()
            _ok(dl, call(dl, max(1, mean * E), E, m, n), f"grouped {mean} rows of {E}")

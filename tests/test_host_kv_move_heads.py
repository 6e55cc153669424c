"""CPU check: a move of a few tokens of as many heads as the checks let through is a
launch that can be made."""

import pytest

from test_host_dryrun import _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import CACHE, SLOTS, UNSUPPORTED, WS

OTHER = 0x1200000000


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,H", [(1, (1 << 22) - 1), (1, 1 << 22), (1, 1 << 27), (32, 1 << 22), (31, (1 << 22) + 1), (512, 1 << 18)])
def test_move_launches(dl, D, n, H):  # noqa: F811
    nb = dl.brq_kv_move_workspace_bytes(n, H, D)
    assert (nb == 0) == (H < 1 << 22)
    dl.brq_dryrun_reset()
    _ok(dl, dl.brq_kv_move(CACHE, SLOTS, OTHER, n, H, D, 16, 3, WS if nb else None, nb, None), f"move of {n} x {H}")
    assert dl.brq_dryrun_launches() == 1
    assert dl.brq_kv_move(CACHE, SLOTS, OTHER, (1 << 27) // H + 1, H, D, 16, 3, WS, 1 << 50, None) == UNSUPPORTED

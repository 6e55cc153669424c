"""CPU check: tree attention over as many units as the checks let through is a
launch that can be made."""

import pytest

from test_host_dryrun import _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import CACHE, LENS, TABLE, WS, X, Y

MASK = 0x1000000000


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,N,hq,H", [(4096, 1, 2048, 2048), (65, 1, 258000, 258000), (4096, 1, 4095, 4095),
                                      (2048, 1, 4095, 4095), (4096, 1, 4088, 511), (4096, 2, 2040, 510), (4095, 64, 64, 64),
                                      (4096, 17, 240, 240), (1 << 20, 1, 15, 15), (70, 1, 200000, 200000)])
def test_tree_launches(dl, D, B, N, hq, H):  # noqa: F811
    nb = dl.brq_tree_attention_workspace_bytes(B, N, hq, H, D)
    dl.brq_dryrun_reset()
    _ok(dl, dl.brq_tree_attention(None, X, hq * D, 1, CACHE, 1000, TABLE, 3, LENS, MASK, B, N, hq, H, D, 16, 0.1, 0, Y,
                                  hq * D, None, WS if nb else None, nb, None), f"tree {B}x{N}, {H} heads of {D}")
    assert dl.brq_dryrun_launches() == 1

"""A move of a few tokens of more heads than one launch has workgroups for."""

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_moves_of_four_million_heads():
    """As its two halves, of which each is one launch, one after the other."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    H, D, P = (1 << 22) + 2, 64, 16
    announce(f"kv move of {H} heads")
    cache = brq.kv_cache(2, H, D, P)
    cache.random_(0, 256)
    src, dst = (torch.tensor(x, device="cuda") for x in ([3, 17, 30, -1, 5], [17, 18, 4, 2, 32]))
    halves = []
    for part in (slice(0, H // 2), slice(H // 2, H)):
        halves.append(brq.kv_move(cache[:, part].contiguous(), src, dst, D, P))
    before = cache[:, ::1000].clone()
    brq.kv_move(cache, src, dst, D, P)
    assert torch.equal(cache[:, :H // 2], halves[0]) and torch.equal(cache[:, H // 2:], halves[1])
    assert not torch.equal(cache[:, ::1000], before)

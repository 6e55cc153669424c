"""Tree attention over more units than one launch could join (2^23 of a head of
256), against the attention of one token."""

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_more_units_than_a_join_can_have():
    import butterfly_rotation_quantization_amd as brq
    import torch
    B, H, D, P = 4096, 2048, 256, 16
    announce(f"tree of {B} x {H} units of heads of {D}")
    assert brq.tree_attention_workspace(B, 1, H, H, D) is None
    torch.manual_seed(1)
    cache = brq.kv_cache(1, H, D, P)  # one page, which all sequences hold
    k, v = (torch.randn((P, H, D), device="cuda") for _ in range(2))
    brq.kv_append(None, k, v, torch.arange(P, device="cuda"), cache, P)
    q = torch.randn((B, 1, H, D), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    ctx = (torch.arange(B, dtype=torch.int32, device="cuda") % 18) - 1  # none to all of the page, past its end
    mask = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    lse = torch.zeros((B, 1, H), device="cuda")
    out = brq.tree_attention(None, q, cache, table, ctx, mask, P, lse=lse)
    one_lse = torch.zeros((B, H), device="cuda")
    one = brq.paged_attention(None, q[:, 0], cache, table, torch.where(ctx < 0, 0, ctx + 1), P, lse=one_lse)
    assert torch.equal(torch.isneginf(lse[:, 0]), torch.isneginf(one_lse))
    # scores within 10 of zero, off by 2 (2^-16 + 2 D 2^-23) of their terms' sum, below 2^8, at most
    fine = torch.isfinite(one_lse)
    assert ((lse[:, 0] - one_lse)[fine].abs() <= 2.0 ** -5).all()
    for b in range(0, B, 256):  # each is the formula's within half a step of bfloat16, and next to nothing
        x, y = out[b:b + 256, 0].float(), one[b:b + 256].float()
        assert (x - y).norm() <= 2.0 ** -7 * y.norm()
    assert not out[ctx < 0].any()

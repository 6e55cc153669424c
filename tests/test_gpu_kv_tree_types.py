"""What the tree attention gives for 16-bit rows is the rounding of what it gives
for the same rows in float32: queries, scores, probabilities and sums have the same bits
whatever the rows' type."""

import numpy as np
import pytest

from gpu_util import announce, to_dev, torch_dtype
from test_gpu_kv import build
from test_gpu_kv_tree import to_mask, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,N,hq,H,window", [(64, 7, 8, 2, 0), (64, 33, 4, 1, 100), (128, 3, 4, 1, 0), (128, 64, 8, 1, 0),
                                             (256, 9, 4, 2, 17)])
def test_16_bit_rows_round_the_float32_result(D, N, hq, H, window, dtype):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"tree {dtype} against float32 D={D} N={N}")
    rng = np.random.default_rng(D + N)
    ctx = [1000, 0, 33, 5000]
    cache, _, table, plan, _, _ = build(rng, [c + N for c in ctx], H, D, 32, True)
    mask = to_dev(to_mask([tree(rng, N) for _ in ctx]), "i64")
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    q = torch.randn((len(ctx), N, hq, D), device="cuda").to(torch_dtype(dtype))
    lse = [torch.empty((len(ctx), N, hq), device="cuda") for _ in range(2)]
    got, want = (brq.tree_attention(plan, x, cache, to_dev(table, "i32"), lens, mask, 32, window=window, lse=y)
                 for x, y in zip((q, q.float()), lse))
    assert torch.equal(got, want.to(q.dtype)) and torch.equal(*lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_an_infinite_value_of_the_context_is_one(D, dtype):
    """Beyond a mask as among the drafts: infinite in its block for every row, also where
    its probability is 1, which has no lower bits; one that is NaN is NaN."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    from oracle import mx as X
    announce(f"tree infinite context D={D} {dtype}")
    rng = np.random.default_rng(D)
    P, H, N, n = 16, 2, 5, 300
    cache, _, table, _, _, slots = build(rng, [n + N], H, D, P, False)
    q = torch.randn((1, N, 4, D), device="cuda").to(torch_dtype(dtype))
    t, lens, mask = to_dev(table, "i32"), torch.tensor([n], dtype=torch.int32, device="cuda"), to_dev(to_mask([tree(rng, N)]), "i64")
    before = brq.tree_attention(None, q, cache, t, lens, mask, P)
    s = int(slots[70])  # in the third step; of head 1, block 1
    for peak in (False, True):
        for byte in (253, 254, 255):
            c = X.Cache.from_bytes(cache.cpu().numpy(), D, P)
            c.vs[s // P, 1, s % P, 1] = byte
            c.vc[s // P, 1, s % P, 16:32] = 0x77  # 6 throughout
            if peak:  # every key of the head scores 0, so that every probability is 1
                c.kc[:, 1] = 0
            out = brq.tree_attention(None, q, to_dev(c.to_bytes(), "u8"), t, lens, mask, P)
            mine = out[0, :, 2:].float()
            assert torch.equal(out[0, :, :2], before[0, :, :2])
            hit = mine[..., 32:64]
            assert torch.isnan(hit).all() if byte == 255 else torch.isposinf(hit).all()
            assert torch.isfinite(mine[..., :32]).all() and torch.isfinite(mine[..., 64:]).all()

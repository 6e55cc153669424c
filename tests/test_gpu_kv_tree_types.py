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

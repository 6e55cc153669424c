"""The tree attention where all scores of a row, of its first keys or of one
wavefront's lie far from zero, against the formula in 64 bits (oracle/mx.py); the
bound is test_gpu_kv_tree.py's."""

import numpy as np
import pytest

from gpu_util import announce, from_dev, to_dev, torch_dtype
from oracle import mx as X
from test_gpu_kv import rht
from test_gpu_kv_tree import check, to_mask, tree

pytestmark = pytest.mark.gpu


def leaning(rng, ctx, N, H, D, P, rot, level):
    """A cache whose keys have u, a vector of signs, as a common component, so that u scores
    level[token] with them (scale 1/sqrt D; the format's rounding spreads this by some units),
    beside ordinary values: cache, oracle, table, plan, M, u."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    used = [(c + N + P - 1) // P for c in ctx]
    order = rng.permutation(sum(used) + 2)
    table = np.full((len(ctx), max(used)), 2 ** 31 - 1, dtype=np.int32)
    u = rng.choice([-1.0, 1.0], D).astype(np.float32)
    cache = torch.full((sum(used) + 2, H, P * (D + D // 16)), 255, dtype=torch.uint8, device="cuda")
    plan, signs = rht(D) if rot else (None, None)
    at = 0
    for b, c in enumerate(ctx):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        n = c + N
        slots = table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        k = rng.standard_normal((n, H, D)).astype(np.float32)
        k += (np.array([level(b, j) for j in range(n)], np.float32) / np.float32(np.sqrt(D)))[:, None, None] * u
        v = rng.standard_normal((n, H, D)).astype(np.float32) + 0.5
        brq.kv_append(plan, to_dev(k, "f32"), to_dev(v, "f32"), to_dev(slots, "i64"), cache, P)
    M = X.hadamard64(D, signs) if rot else None
    return cache, X.Cache.from_bytes(cache.cpu().numpy(), D, P), table, plan, M, u


def attend(ctx, N, hq, H, D, P, rot, dtype, level, window=0, mask=None, seed=0):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"tree far ctx={list(ctx)[:5]} N={N} hq={hq} D={D} {dtype} window={window}")
    rng = np.random.default_rng(seed + D + N)
    cache, ref, table, plan, M, u = leaning(rng, ctx, N, H, D, P, rot, level)
    q = torch.from_numpy((u + 0.25 * rng.standard_normal((len(ctx), N, hq, D))).astype(np.float32)).to(torch_dtype(dtype)).cuda()
    mask = to_mask([tree(rng, N) for _ in ctx] if mask is None else mask)
    lens, lse = np.array(ctx, np.int32), torch.full((len(ctx), N, hq), 7.0, device="cuda")
    out = brq.tree_attention(plan, q, cache, to_dev(table, "i32"), to_dev(lens, "i32"), to_dev(mask, "i64"), P,
                             window=window, lse=lse)
    want, wlse, slack = X.tree_attention(from_dev(q), ref, table, lens, mask, D ** -0.5, window, M)
    check(from_dev(out), from_dev(lse), want, wlse, slack, lens, D, dtype)
    return wlse


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,rot", [(64, False), (128, True), (256, False)])
@pytest.mark.parametrize("level", [-95.0, -200.0, -1000.0, 200.0])
def test_all_scores_far_from_zero(D, rot, dtype, level):
    """No key, one, some beyond a step's, those of several workgroups."""
    lse = attend([0, 1, 33, 700], 5, 8, 2, D, 32, rot, dtype, lambda b, j: level)
    assert (lse < -50).all() if level < 0 else (lse > 100).all()


@pytest.mark.parametrize("window", [1, 7, 33])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_windows_of_low_scores(D, window):
    attend([0, 2, 31, 64, 300], 6, 4, 1, D, 16, True, "f32", lambda b, j: -250.0, window=window)


def test_one_visible_key_that_scores_low():
    """Single drafts, of empty contexts and behind a window's edge, in either column tile."""
    for N in (1, 40):
        own = [[1 << j for j in range(N)]] * 3
        attend([0, 0, 16], N, 3, 1, 128, 16, False, "bf16", lambda b, j: -300.0, window=1, mask=own)
        attend([0, 0, 0], N, 3, 1, 64, 16, True, "f32", lambda b, j: -300.0, mask=own)


@pytest.mark.parametrize("D,ctx,N", [(128, 600, 5), (64, 20011, 33), (256, 9000, 3), (128, 20011, 64)])
def test_low_scores_of_one_wavefront(D, ctx, N):
    """The 32 keys that a wavefront begins with score low, the others as usual; then all but an early key do."""
    attend([ctx], N, 4, 1, D, 64, False, "f32", lambda b, j: -300.0 if 32 <= j < 64 else 0.0)
    attend([ctx], N, 4, 1, D, 64, True, "bf16", lambda b, j: 60.0 if j == 5 else -200.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_chain_of_low_scores_is_what_single_tokens_give(dtype):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"tree chain far {dtype}")
    rng = np.random.default_rng(4)
    N, D, P, H, hq, ctx = 4, 128, 32, 2, 8, [100, 3, 700]
    cache, ref, table, plan, M, u = leaning(rng, ctx, N, H, D, P, True, lambda b, j: -200.0)
    q = torch.from_numpy((u + 0.25 * rng.standard_normal((3, N, hq, D))).astype(np.float32)).to(torch_dtype(dtype)).cuda()
    t, lens = to_dev(table, "i32"), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    rows = to_mask([[2 ** (i + 1) - 1 for i in range(N)]] * 3)
    out = brq.tree_attention(plan, q, cache, t, lens, to_dev(rows, "i64"), P)
    _, _, (spread, terms) = X.tree_attention(from_dev(q), ref, table, ctx, rows, D ** -0.5, 0, M)
    # both differ from the formula by the bound's share of scores and sums, and by their rounding
    rel = 2 * (2.0 ** -16 + 2 * D * 2.0 ** -23) * terms + 2.0 ** -16 + 120 * 2.0 ** -23
    step = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7}[dtype]
    for i in range(N):
        one = from_dev(brq.paged_attention(plan, q[:, i].contiguous(), cache, t, lens + i + 1, P))
        bound = 4 * rel[:, i, :, None] * spread[:, i] + step * np.abs(one) + 2.0 ** -24
        assert (np.abs(from_dev(out[:, i]) - one) <= bound).all()

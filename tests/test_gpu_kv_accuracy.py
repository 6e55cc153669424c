"""How exact the attention's scores and normaliser are, whatever the queries'
type: its log-sum-exp is a float32 output, and is compared with 64 bits.

A score's error, from the parts of the computation: the query's scaling rounds
once and the factor itself once (2^-24 each); a query in pieces keeps 2^-23 of
the largest entry of its block of 32, so the score loses at most 2^-23 of the
sum of |k_j| times that entry (a factor of two is allowed for it); at most eight
products of 128 values and one addition each round or truncate a sum (2^-23
each), and the unit a term or two inside a product: 16 times 2^-23 of the sum of
|q_j k_j| covers all.  A transform ahead of it adds log2 D + 2 roundings, 2^-24
sqrt(D) of its largest entry each.  lse then is at most the largest score error
off, plus 2^-21 of itself and of one for the exponentials, sums and logarithm."""

import numpy as np
import pytest

from gpu_util import announce, to_dev, torch_dtype
from oracle import mx as X
from test_gpu_kv import build, rht

pytestmark = pytest.mark.gpu


def block_top(x):
    """Each entry's block's largest magnitude (blocks of 32 on the last axis)."""
    b = np.abs(x).reshape(*x.shape[:-1], -1, 32)
    return np.repeat(b.max(-1), 32, axis=-1)


def score_bound(q, k):
    """Bound of the scores' error: q [heads, D], k [keys, D], both as they enter."""
    return 16 * 2.0 ** -23 * (np.abs(q) @ np.abs(k).T) + 2.0 ** -22 * (block_top(q) @ np.abs(k).T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spread", [0, 8])
def test_a_score_of_mixed_codes(D, dtype, spread):
    """One key, so that lse is its score: its largest codes beside small ones,
    its blocks' scales 2^spread and more apart, against queries of widely
    different entries."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention score of mixed codes D={D} {dtype} spread={spread}")
    rng = np.random.default_rng(D + spread)
    for heads in (8, 16):  # one and two column tiles
        k = rng.choice([0.5, 1.0, 1.5], (1, 1, D)).astype(np.float32)
        k[..., 3::32] = 6.0
        k *= np.exp2(rng.integers(-spread, spread + 1, D // 32)).repeat(32).astype(np.float32)
        cache, at = brq.kv_cache(1, 1, D, 16), torch.zeros(1, dtype=torch.int64, device="cuda")
        brq.kv_append(None, to_dev(k, "f32"), to_dev(k, "f32"), at, cache, 16)
        key = X.Cache.from_bytes(cache.cpu().numpy(), D, 16).keys_values()[0][0, 0, :1]
        assert np.array_equal(key[0], k[0, 0])  # exact in the format
        q = rng.choice([-1.0, 1.0], (64, heads, D)) * np.exp2(rng.uniform(-16, 0, (64, heads, D)))
        q[..., 3::32] = 1.99
        q[32:] *= np.exp2(rng.integers(-spread, spread + 1, (32, heads, D // 32))).repeat(32, axis=-1) * 2.0 ** -6
        q = torch.from_numpy(q.astype(np.float32)).to(torch_dtype(dtype)).cuda()
        lse = torch.empty((64, heads), device="cuda")
        zeros = torch.zeros((64, 1), dtype=torch.int32, device="cuda")
        brq.paged_attention(None, q, cache, zeros, zeros[:, 0] + 1, 16, scale=1.0, lse=lse)
        qh = q.double().cpu().numpy().reshape(-1, D)
        want = (qh @ key.T)[:, 0]
        off = np.abs(lse.double().cpu().numpy().reshape(-1) - want)
        bound = score_bound(qh, key)[:, 0] + 2.0 ** -21 * (1 + np.abs(want))
        assert (off <= bound).all(), f"{(off / bound).max():.1f} times the bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,rot,scale", [(64, False, None), (128, False, None), (128, True, None), (256, True, None),
                                         (128, False, 6.0)])
def test_log_sum_exp(D, rot, scale, dtype):
    """Over many keys, also with scores in the hundreds: the normaliser is a sum
    of float32 probabilities."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention lse D={D} rot={rot} {dtype} scale={scale}")
    rng = np.random.default_rng(D + rot)
    lens, hq, H, P = [1, 33, 700, 5000], 16, 2, 64
    scale = D ** -0.5 if scale is None else scale
    cache, ref, table, plan, M, _ = build(rng, lens, H, D, P, rot)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, D)).astype(np.float32)).to(torch_dtype(dtype)).cuda()
    lse = torch.empty((len(lens), hq), device="cuda")
    brq.paged_attention(plan, q, cache, to_dev(table, "i32"), torch.tensor(lens, dtype=torch.int32).cuda(), P,
                        scale=scale, lse=lse)
    K, _ = ref.keys_values()
    got = lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        j = np.arange(n)
        for h in range(H):
            k = K[table[b, j // P], h, j % P]
            x = q[b, h * 8:h * 8 + 8].double().cpu().numpy()
            x = x if M is None else x @ M.T
            s = scale * (x @ k.T)
            top = s.max(1, keepdims=True)
            want = top[:, 0] + np.log(np.exp(s - top).sum(1))
            err = abs(scale) * score_bound(x, k)
            if M is not None:
                first = np.linalg.norm(x, axis=1, keepdims=True)  # no entry of a sum on the way is larger
                err += abs(scale) * (np.log2(D) + 2) * 2.0 ** -24 * first * np.abs(k).sum(1)
            # keys that hold next to nothing of the sum do not matter
            err = np.where(s > top - 40, err, 0).max(1)
            bound = err + 2.0 ** -21 * (1 + np.abs(want))
            off = np.abs(got[b, h * 8:h * 8 + 8] - want)
            assert (off <= bound).all(), f"sequence {b}, head {h}: {(off / bound).max():.1f} times the bound"

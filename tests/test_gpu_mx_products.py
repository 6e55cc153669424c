"""The product on every kernel's path, compared where it can be bit for bit.

With scales of two neighbouring powers of two every product is a multiple of
1/16 and every sum of them, in whatever order, stays below 2^24 sixteenths (n
products of at most 36 are 2^24 sixteenths at n = 29127, all of one sign), so
float32 sums are exact and the result has to be the formula's, rounded once.

With wide scales sums round: a product of n takes n / 64 additions at most, each
within 2^-23 of the partial sum, whose norm over the outputs is taken to be
below twice the result's.  In the norm the error is then below (n / 32 + 8)
2^-23 of the result's norm, 2^-14 at the longest; partial sums of 16 bits
would be off by 2^-9."""

import numpy as np
import pytest

from gpu_util import announce, torch_dtype
from oracle import mx as X
from test_gpu_mx import SHAPES, operands

pytestmark = pytest.mark.gpu

# (T, m, n) and the parts of n that the sums are made in, as the workspace's size shows
MORE = [
    (2048, 4096, 512, 1), (2047, 4093, 544, 1), (1500, 5000, 256, 1),  # up to 512 tiles of 128: two stages in LDS
    (100, 130, 8224, 4), (65, 513, 16416, 8), (300, 385, 16640, 8),    # many parts, odd widths, ragged last stages
    (129, 1022, 65536, 16), (70, 64, 22528, 11),
    (40, 16384, 8192, 2), (64, 8192, 16384, 4),                         # up to 64 tokens over a wide weight
]


def on_gpu(pair):
    import torch
    return [torch.from_numpy(z).cuda() for z in pair]


def values64(codes, scales):
    """X.values, on the GPU."""
    import torch
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    mag = torch.from_numpy(np.concatenate((X.MAGNITUDES, -X.MAGNITUDES))).cuda()
    s = torch.pow(torch.full(scales.shape, 2.0, dtype=torch.float64, device="cuda"), scales.double() - 127)
    return mag[c] * s.repeat_interleave(32, dim=-1)


def product64(a, b):
    return values64(*a) @ values64(*b).t().contiguous()


def parts_of(T, m, n):
    """Parts of the long axis, from the workspace beyond the scales' images of 128 x 128 tiles."""
    import butterfly_rotation_quantization_amd as brq
    ws = brq.mx_matmul_workspace(T, m, n)
    images = (-(-T // 128) + -(-m // 128)) * -(-n // 256) * 8 * 128
    return max(1, (ws.numel() - images) // (4 * T * m))


@pytest.mark.parametrize("T,m,n", SHAPES + [s[:3] for s in MORE])
def test_exact_sums(T, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    rng = np.random.default_rng(T * 7 + m + n)
    assert 36 * 16 * n < 2 ** 24 or n > 29127
    a, b = [on_gpu(z) for z in operands(rng, T, m, n, 126, 128)]
    want = product64(a, b)
    if n > 29127:  # longer: exact all the same if magnitudes say so
        assert (values64(*a).abs() @ values64(*b).abs().t().contiguous()).max() * 16 < 2 ** 24
    for dtype, pad in (("f32", 0), ("f32", 3), ("bf16", 1), ("f16", 0)):
        announce(f"mx exact product {T}x{m}x{n} {dtype} pad={pad}")
        y = torch.full((T, m + pad), 7.0, dtype=torch_dtype(dtype), device="cuda")
        brq.mx_matmul(*a, *b, y=y[:, :m])
        assert torch.equal(y[:, :m], want.float().to(torch_dtype(dtype))), f"{int((y[:, :m] != want).sum())} differ"
        assert (y[:, m:] == 7).all()


@pytest.mark.parametrize("T,m,n,parts", MORE)
def test_the_paths_meant_here_are_taken(T, m, n, parts):
    assert parts_of(T, m, n) == parts


@pytest.mark.parametrize("T,m,n", SHAPES + [s[:3] for s in MORE])
def test_sums_of_wide_scales_in_the_norm(T, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx product norm {T}x{m}x{n}")
    rng = np.random.default_rng(T + m * 3 + n)
    a, b = [on_gpu(z) for z in operands(rng, T, m, n, 110, 140)]
    want = product64(a, b)
    got = brq.mx_matmul(*a, *b, out_dtype=torch.float32).double()
    assert (got - want).norm() <= (n / 32 + 8) * 2.0 ** -23 * want.norm()


@pytest.mark.parametrize("T", [1, 20, 65])
def test_rows_beyond_2_to_the_23(T):
    """The few blocks that are not zero lie at both ends and about the middle."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    m, nb = 3, (1 << 18) + 5
    n = 32 * nb
    announce(f"mx product {T}x{m}x{n}")
    rng = np.random.default_rng(T)
    at = np.array([0, 1, 2, 7, 12345, nb // 2, (1 << 18) - 1, 1 << 18, nb - 3, nb - 1])
    small = operands(rng, T, m, 32 * len(at), 126, 128)
    big = []
    for (codes, scales), rows in zip(small, (T, m)):
        c = torch.zeros((rows, nb, 16), dtype=torch.uint8, device="cuda")
        s = torch.full((rows, nb), 127, dtype=torch.uint8, device="cuda")
        c[:, torch.from_numpy(at)] = torch.from_numpy(codes.reshape(rows, len(at), 16)).cuda()
        s[:, torch.from_numpy(at)] = torch.from_numpy(scales).cuda()
        big.append((c.view(rows, n // 2), s))
    y = brq.mx_matmul(*big[0], *big[1], out_dtype=torch.float32)
    assert torch.equal(y.double(), product64(*[on_gpu(z) for z in small]))

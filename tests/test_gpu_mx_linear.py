"""The product with an epilogue, on every kernel's path: sums that are exact in
float32 whatever their order (scales of two neighbouring powers of two), so that
what is compared is the epilogue alone, against the formula in 64 bits
(oracle/mx.py, whose bound counts float32's roundings).  The output adds half a
step of its type, or half of float16's smallest."""

import numpy as np
import pytest

from gpu_util import announce, from_dev, to_dev, torch_dtype
from oracle import mx as X
from test_gpu_mx import operands
from test_gpu_mx_products import on_gpu

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}
# one and two tiles of outputs, both streams, tiles of 128 (two and three stages in LDS; parts) and of 256, rows too short
SHAPES = [(1, 1, 32), (1, 4096, 4096), (7, 259, 160), (16, 11008, 4000), (17, 64, 1024), (33, 48, 8192), (64, 512, 512),
          (50, 8193, 544), (128, 256, 1376), (257, 770, 288), (65, 513, 16416), (300, 384, 16640), (2100, 4200, 544),
          (2101, 4197, 768), (2048, 4096, 512), (100, 70, 160), (9, 8200, 32)]
PARTS = ["bias", "act", "mul", "residual"]


def operand(rng, shape, dtype, gap):
    """A device tensor of normal values whose rows are `gap` elements apart, and its values."""
    import torch
    t = torch.from_numpy(rng.standard_normal((*shape[:-1], shape[-1] + gap)).astype(np.float32))
    t = t.to(torch_dtype(dtype)).cuda()[..., :shape[-1]]
    return t, from_dev(t)


def scaled(rng, T, m, n):
    """Operands whose products' sums are about 1 to 5, all multiples of 2^-k and exact in float32."""
    e = 127 - int(np.log2(n)) // 4
    return operands(rng, T, m, n, e - 1, e + 1)


def sums(a, b):
    """The product in 64 bits: exact, as are the values (by ldexp: a power function's last bit would show where a
    sum is zero)."""
    import torch
    x, w = (torch.from_numpy(X.values(*z)).cuda() for z in (a, b))
    return (x @ w.t().contiguous()).cpu().numpy()


def check(got, want, err, dtype):
    bound = err + HALF[dtype] * (np.abs(want) + err) + TINY[dtype]
    over = ~(np.abs(got - want) <= bound)
    assert not over.any(), f"{int(over.sum())} of {over.size}, first {np.argwhere(over)[:3].tolist()}: " \
                           f"{got[over][:3]} for {want[over][:3]}, bound {bound[over][:3]}"


@pytest.mark.parametrize("T,m,n", SHAPES)
def test_linear(T, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    rng = np.random.default_rng(T + 3 * m + n)
    a, b = scaled(rng, T, m, n)
    ad, bd = on_gpu(a), on_gpu(b)
    s = sums(a, b)
    cases = [("gelu", "f32", "bf16", 0, {"bias", "act", "mul", "residual"}), ("silu", "bf16", "f16", 4, {"act", "mul"}),
             ("gelu_tanh", "f16", "f32", 3, {"bias", "act"}), (None, "bf16", "bf16", 8, {"residual"}),
             ("relu", "f32", "f32", 5, {"bias", "act", "residual"})]
    for act, dtype, other, gap, parts in cases:
        announce(f"mx linear {T}x{m}x{n} {act} {dtype} {sorted(parts)} gap {gap}")
        (bias, bh), = [operand(rng, (m,), other, 0)]
        (mul, mh), (res, rh) = (operand(rng, (T, m), other, gap) for _ in range(2))
        y = torch.full((T, m + gap), 7.0, dtype=torch_dtype(dtype), device="cuda")
        brq.mx_linear(*ad, *bd, bias=bias if "bias" in parts else None, act=act, mul=mul if "mul" in parts else None,
                      residual=res if "residual" in parts else None, y=y[:, :m])
        want, err = X.epilogue(s, bh if "bias" in parts else None, act, mh if "mul" in parts else None,
                               rh if "residual" in parts else None)
        check(from_dev(y[:, :m]), want, err, dtype)
        assert (y[:, m:] == 7).all()


@pytest.mark.parametrize("T,m,n", [(1, 300, 4096), (40, 257, 512), (300, 384, 16640), (300, 1100, 768)])
def test_the_output_may_be_an_operand(T, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx linear in place {T}x{m}x{n}")
    rng = np.random.default_rng(T)
    ad, bd = (on_gpu(x) for x in scaled(rng, T, m, n))
    mul, res = (operand(rng, (T, m), "bf16", 0)[0] for _ in range(2))
    want = brq.mx_linear(*ad, *bd, act="silu", mul=mul, residual=res)
    for y, kw in ((mul.clone(), "mul"), (res.clone(), "residual")):
        brq.mx_linear(*ad, *bd, act="silu", **{"mul": mul, "residual": res, kw: y}, y=y)
        assert torch.equal(y, want), kw


@pytest.mark.parametrize("T,m,n", [(3, 64, 256), (40, 520, 544), (128, 300, 1376), (300, 384, 16640)])
def test_without_parts_it_is_the_product(T, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx linear plain {T}x{m}x{n}")
    rng = np.random.default_rng(T)
    ad, bd = (on_gpu(x) for x in operands(rng, T, m, n, 100, 140))
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(brq.mx_linear(*ad, *bd, out_dtype=dtype), brq.mx_matmul(*ad, *bd, out_dtype=dtype))
        bias = torch.zeros(m, device="cuda")
        assert torch.equal(brq.mx_linear(*ad, *bd, bias=bias, out_dtype=dtype), brq.mx_matmul(*ad, *bd, out_dtype=dtype))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_over_their_range(act):
    """Sums of zero (a matrix of zeros), so that the bias is what the activation sees: to both ends of float32."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx linear activation {act}")
    x = np.concatenate([np.linspace(-12, 12, 4001), np.geomspace(1e-30, 3e38, 500), -np.geomspace(1e-30, 3e38, 500),
                        [0.0, -0.0]]).astype(np.float32)
    m = len(x)
    zero = lambda r: (torch.zeros((r, 16), dtype=torch.uint8, device="cuda"),  # noqa: E731
                      torch.full((r, 1), 127, dtype=torch.uint8, device="cuda"))
    bias = torch.cat((torch.from_numpy(x), torch.tensor([float("nan"), float("inf")]))).cuda()
    y = from_dev(brq.mx_linear(*zero(1), *zero(m + 2), bias=bias, act=act, out_dtype=torch.float32))[0]
    want, err = X.activation(x.astype(np.float64), act)
    fine = np.abs(want) < 1e38
    check(y[:m][fine], want[fine], (err * 2.0 ** -24 + 2e-38)[fine], "f32")
    assert np.isnan(y[m]) and np.isposinf(y[m + 1])


def apart(rows, m, dtype, over=33):
    """Rows so far apart that the last one's elements lie beyond 2^`over` bytes."""
    import torch
    size = torch.empty((), dtype=dtype).element_size()
    ld = (2 ** over // size // max(rows - 1, 1) + m + 16) // 16 * 16
    return torch.empty((rows - 1) * ld + m, dtype=dtype, device="cuda").as_strided((rows, m), (ld, 1))


@pytest.mark.parametrize("T,m,n", [(20, 70, 160), (300, 384, 16640), (300, 520, 512), (2101, 4197, 768), (100, 70, 160)])
def test_rows_beyond_32_bit_offsets(T, m, n):
    """Output, factor and residual whose rows are gigabytes away, against rows next to each other."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx linear {T}x{m}x{n} far apart")
    rng = np.random.default_rng(m)
    a, b = (on_gpu(z) for z in scaled(rng, T, m, n))
    mul, res = torch.randn((T, m), device="cuda").half(), torch.randn((T, m), device="cuda")
    far = apart(T, m, torch.float16), apart(T, m, torch.float32), apart(T, m, torch.bfloat16)
    far[0].copy_(mul), far[1].copy_(res), far[2].zero_()
    want = brq.mx_linear(*a, *b, act="silu", mul=mul, residual=res)
    assert torch.equal(brq.mx_linear(*a, *b, act="silu", mul=far[0], residual=far[1], y=far[2]), want)


def test_linear_empty_sizes():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("mx linear empty sizes")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bias = torch.arange(5, device="cuda", dtype=torch.float32) - 2
    y = brq.mx_linear(u8(3, 0), u8(3, 0), u8(5, 0), u8(5, 0), bias=bias, act="relu", out_dtype=torch.float32)
    assert torch.equal(y, bias.clamp(min=0).expand(3, 5))  # no term: the bias is the sum
    assert brq.mx_linear(u8(0, 16), u8(0, 1), u8(5, 16), u8(5, 1), bias=bias).shape == (0, 5)
    assert brq.mx_linear(u8(3, 16), u8(3, 1), u8(0, 16), u8(0, 1), act="silu").shape == (3, 0)


def test_linear_refusals():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("mx linear refusals")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    ops = (u8(4, 32), u8(4, 2), u8(6, 32), u8(6, 2))
    for bad in (dict(act="tanh"), dict(bias=f(5)), dict(bias=f(6, t=torch.float64)), dict(bias=f(6).cpu()),
                dict(bias=f(12)[::2]), dict(mul=f(4, 5)), dict(mul=f(4, 12)[:, ::2]), dict(residual=f(6)),
                dict(residual=f(4, 6, t=torch.int32)), dict(y=f(4, 5))):
        with pytest.raises(ValueError):
            brq.mx_linear(*ops, **bad)

"""Products grouped by expert, against the formula in 64 bits: operands whose
sums are exact in float32 whatever their order (test_gpu_mx_linear.py), so that
without an epilogue a result is the formula's, rounded once, bit for bit."""

import numpy as np
import pytest

from gpu_util import announce, from_dev, to_dev, torch_dtype
from oracle import mx as X
from test_gpu_mx import operands
from test_gpu_mx_linear import apart, check, operand, scaled, sums
from test_gpu_mx_products import on_gpu

pytestmark = pytest.mark.gpu


def ends(counts, before=0):
    return np.cumsum([before, *counts]).astype(np.int32)


def experts(rng, E, T, m, n):
    """Activations and the weights of E experts."""
    a, b = scaled(rng, T, E * m, n)
    return a, tuple(z.reshape(E, m, -1) for z in b)


def expected(a, b, offsets, T, m):
    """(sums [T, m], the group of each row, -1 for none)."""
    s, of = np.zeros((T, m)), np.full(T, -1)
    offsets = np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, T))
    for e in range(len(offsets) - 1):
        lo, hi = (int(x) for x in offsets[e:e + 2])
        if hi > lo:
            s[lo:hi] = sums([z[lo:hi] for z in a], [z[e] for z in b])
            of[lo:hi] = e
    return s, of


# (rows of each expert, m, n); every row with none, one, a few; one tile and more; ragged everything
SHAPES = [([1], 1, 32), ([0, 3, 0, 1], 70, 160), ([5, 0, 11], 257, 4096), ([1] * 70, 48, 352), ([16, 17, 15, 33], 513, 544),
          ([0] * 130 + [9] + [0] * 5 + [40], 64, 256), ([64, 65, 200, 1], 385, 1376), ([300, 0, 513, 128], 770, 768),
          ([2, 1, 1], 4100, 8192), ([257, 1, 511], 130, 64), ([700, 20, 3, 256], 1030, 2080), ([129, 255, 64], 384, 16640),
          ([40] * 30, 130, 288), ([90] * 20, 600, 512), ([24, 8, 40, 56], 8200, 1056)]


@pytest.mark.parametrize("counts,m,n", SHAPES)
def test_grouped(counts, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    rng = np.random.default_rng(sum(counts) + 3 * m + n)
    E, before, behind = len(counts), 3, 5  # rows of no group at both ends
    offsets = ends(counts, before)
    T = int(offsets[-1]) + behind
    a, b = experts(rng, E, T, m, n)
    ad, bd, off = on_gpu(a), on_gpu(b), to_dev(offsets, "i32")
    s, of = expected(a, b, offsets, T, m)
    mine = of >= 0
    for dtype, pad in (("f32", 0), ("bf16", 5), ("f16", 4)):
        announce(f"mx grouped {counts[:6]} x {m} x {n} {dtype}")
        y = torch.full((T, m + pad), 7.0, dtype=torch_dtype(dtype), device="cuda")
        brq.mx_grouped_matmul(*ad, *bd, off, y=y[:, :m])
        want = torch.from_numpy(s).to(y.dtype).cuda()
        assert torch.equal(y[mine, :m], want[mine])
        assert (y[~mine] == 7).all() and (y[:, m:] == 7).all()
    for act, dtype, other, gap, parts in (("silu", "bf16", "f16", 4, {"act", "mul"}),
                                          ("gelu", "f32", "bf16", 3, {"bias", "act", "mul", "residual"}),
                                          (None, "f16", "f32", 0, {"bias", "residual"})):
        announce(f"mx grouped {counts[:6]} x {m} x {n} {act} {dtype} {sorted(parts)}")
        bias, bh = operand(rng, (E, m), other, 0)
        (mul, mh), (res, rh) = (operand(rng, (T, m), other, gap) for _ in range(2))
        y = torch.full((T, m + gap), 7.0, dtype=torch_dtype(dtype), device="cuda")
        brq.mx_grouped_matmul(*ad, *bd, off, bias=bias if "bias" in parts else None, act=act,
                              mul=mul if "mul" in parts else None, residual=res if "residual" in parts else None,
                              y=y[:, :m])
        want, err = X.epilogue(s[mine], bh[of[mine]] if "bias" in parts else None, act,
                               mh[mine] if "mul" in parts else None, rh[mine] if "residual" in parts else None)
        got = from_dev(y)
        check(got[mine][:, :m], want, err, dtype)
        assert (got[~mine] == 7).all() and (got[:, m:] == 7).all()


@pytest.mark.parametrize("T,m,n", [(40, 130, 288), (700, 300, 1376)])
def test_offsets_beyond_the_rows(T, m, n):
    """What lies outside [0, T] counts as the nearer end, an offset below an earlier one as that."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped offsets outside {T}x{m}x{n}")
    rng = np.random.default_rng(T)
    a, b = experts(rng, 3, T, m, n)
    ad, bd = on_gpu(a), on_gpu(b)
    third = T // 3
    for offsets in ([-5, third, 2 * third, T + 9], [-2 ** 31, 0, third, 2 ** 31 - 1], [T, T, T, T], [0, T, T, T],
                    [third, third, third, third], [T + 1, T + 2, T + 3, T + 4], [5, 3, 4, 4], [0, T, 0, T],
                    [third, 0, T, 0], [T, 0, T, 0], [0, T, -1, -2 ** 31]):
        off = np.array(offsets, dtype=np.int32)
        y = torch.full((T, m), 7.0, device="cuda")
        brq.mx_grouped_matmul(*ad, *bd, to_dev(off, "i32"), y=y)
        s, of = expected(a, b, offsets, T, m)
        got = from_dev(y)
        assert np.array_equal(got[of >= 0], s[of >= 0].astype(np.float32)) and (got[of < 0] == 7).all(), offsets


@pytest.mark.parametrize("E", [70, 200])
def test_many_offsets_in_disorder(E):
    """Offsets at random, as of a table that was never written: every row once at most, whichever wavefront's 64 it falls to."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped offsets in disorder E={E}")
    rng = np.random.default_rng(E)
    for T, m, n in ((60, 40, 96), (40 * E, 130, 256)):
        a, b = experts(rng, E, T, m, n)
        ad, bd = on_gpu(a), on_gpu(b)
        for lo, hi in ((0, T + 1), (-2 ** 31, 2 ** 31 - 1), (T // 2, T // 2 + 9)):
            off = rng.integers(lo, hi, E + 1).astype(np.int32)
            if hi == T + 1:
                off[:E // 2] = np.sort(off[:E // 2]) // 4
            y = torch.full((T, m), 7.0, device="cuda")
            brq.mx_grouped_matmul(*ad, *bd, to_dev(off, "i32"), y=y)
            s, of = expected(a, b, off, T, m)
            got = from_dev(y)
            assert np.array_equal(got[of >= 0], s[of >= 0].astype(np.float32)) and (got[of < 0] == 7).all()


@pytest.mark.parametrize("counts", [[5, 7, 4], [70, 3, 200], [300, 290, 310]])
def test_groups_are_kept_apart(counts):
    """A NaN row, a NaN weight row and a NaN expert show where they belong and nowhere else."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped NaN {counts}")
    rng = np.random.default_rng(sum(counts))
    m, n = 270, 416
    offsets = ends(counts)
    T = int(offsets[-1])
    a, b = experts(rng, 3, T, m, n)
    for z, at in ((a, (counts[0] - 1,)), (b, (0, m - 1)), (b, (2, 0))):
        z[1][(*at, 3)] = 255
        z[0][at][48:64] = 0
    y = from_dev(brq.mx_grouped_matmul(*on_gpu(a), *on_gpu(b), to_dev(offsets, "i32"), out_dtype=torch.float32))
    want = np.zeros((T, m), bool)
    want[counts[0] - 1] = True
    want[:counts[0], m - 1] = True
    want[offsets[2]:, 0] = True
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("T,E", [(24, 8), (600, 4)])
def test_grouped_graph_replays_with_other_groups(T, E):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped graph T={T}")
    rng = np.random.default_rng(T)
    m, n = 264, 1056
    a, b = experts(rng, E, T, m, n)
    ad, bd = on_gpu(a), on_gpu(b)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = T
    y = torch.zeros((T, m), device="cuda")
    ws = brq.mx_grouped_matmul_workspace(T, E, m, n)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        brq.mx_grouped_matmul(*ad, *bd, off, y=y, ws=ws)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            brq.mx_grouped_matmul(*ad, *bd, off, y=y, ws=ws)
    torch.cuda.synchronize()
    for seed in range(4):
        cut = np.sort(np.random.default_rng(seed).integers(0, T + 1, E - 1))
        off.copy_(torch.from_numpy(np.array([0, *cut, T], dtype=np.int32)))
        if ws is not None:
            ws.fill_(255)  # nothing is kept in it
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, brq.mx_grouped_matmul(*ad, *bd, off, out_dtype=torch.float32)), seed


@pytest.mark.parametrize("rows", [5, 100])
def test_weights_beyond_32_bit_offsets(rows):
    """Rows of the first and the last of 64 experts, whose weights take 4.6 GB, against each expert alone."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped 64 experts of 16384 x 8192, {rows} rows")
    E, m, n = 64, 16384, 8192
    rng = np.random.default_rng(rows)
    (a, b), T = scaled(rng, 2 * rows, 2 * m, n), 2 * rows
    (ac, asc), (bc, bsc) = on_gpu(a), on_gpu(b)
    codes = torch.full((E, m, n // 2), 0x77, dtype=torch.uint8, device="cuda")
    scales = torch.full((E, m, n // 32), 255, dtype=torch.uint8, device="cuda")
    for e, i in ((0, 0), (E - 1, 1)):
        codes[e], scales[e] = bc[i * m:(i + 1) * m], bsc[i * m:(i + 1) * m]
    off = torch.full((E + 1,), rows, dtype=torch.int32, device="cuda")
    off[0], off[E] = 0, T
    y = brq.mx_grouped_matmul(ac, asc, codes, scales, off, out_dtype=torch.float32)
    for i in range(2):
        r, w = slice(i * rows, (i + 1) * rows), slice(i * m, (i + 1) * m)
        assert torch.equal(y[r], brq.mx_matmul(ac[r].contiguous(), asc[r].contiguous(), bc[w].contiguous(), bsc[w].contiguous(),
                                               out_dtype=torch.float32))


@pytest.mark.parametrize("counts,m,n", [([3, 0, 1, 2], 70, 160), ([300, 0, 513, 128], 770, 768), ([40, 41, 39], 130, 288)])
def test_grouped_rows_beyond_32_bit_offsets(counts, m, n):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"mx grouped {counts} {m}x{n} far apart")
    rng, T = np.random.default_rng(m), sum(counts)
    a, b = experts(rng, len(counts), T, m, n)
    off = to_dev(ends(counts), "i32")
    mul, res = torch.randn((T, m), device="cuda").half(), torch.randn((T, m), device="cuda")
    far = apart(T, m, torch.float16), apart(T, m, torch.float32), apart(T, m, torch.bfloat16)
    far[0].copy_(mul), far[1].copy_(res), far[2].zero_()
    want = brq.mx_grouped_matmul(*on_gpu(a), *on_gpu(b), off, act="silu", mul=mul, residual=res)
    assert torch.equal(brq.mx_grouped_matmul(*on_gpu(a), *on_gpu(b), off, act="silu", mul=far[0], residual=far[1], y=far[2]), want)


def test_one_group_is_the_linear_product():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("mx grouped of one")
    rng = np.random.default_rng(2)
    for T, m, n in ((1, 300, 4096), (50, 257, 512), (300, 520, 1376)):
        ad, bd = (on_gpu(x) for x in scaled(rng, T, m, n))
        off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        one = brq.mx_grouped_matmul(*ad, *(z[None] for z in bd), off, act="silu")
        assert torch.equal(one, brq.mx_linear(*ad, *bd, act="silu"))


def test_grouped_empty_sizes_and_refusals():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("mx grouped empty sizes, refusals")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    bias = torch.arange(10, device="cuda", dtype=torch.float32).view(2, 5) - 4
    y = brq.mx_grouped_matmul(u8(3, 0), u8(3, 0), u8(2, 5, 0), u8(2, 5, 0), i32(0, 1, 3), bias=bias, act="relu",
                              out_dtype=torch.float32)
    assert torch.equal(y, bias[[0, 1, 1]].clamp(min=0))
    assert brq.mx_grouped_matmul(u8(0, 16), u8(0, 1), u8(2, 5, 16), u8(2, 5, 1), i32(0, 0, 0)).shape == (0, 5)
    assert brq.mx_grouped_matmul(u8(3, 16), u8(3, 1), u8(2, 0, 16), u8(2, 0, 1), i32(0, 1, 3)).shape == (3, 0)
    y = f(3, 5) + 7
    assert (brq.mx_grouped_matmul(u8(3, 16), u8(3, 1), u8(0, 5, 16), u8(0, 5, 1), i32(0), y=y) == 7).all()  # no group
    ops = (u8(4, 32), u8(4, 2), u8(2, 6, 32), u8(2, 6, 2), i32(0, 2, 4))
    for i, bad in ((4, i32(0, 4)), (4, i32(0, 2, 4).long()), (4, i32(0, 2, 4).cpu()), (2, u8(6, 32)), (2, u8(2, 6, 30)),
                   (3, u8(2, 5, 2)), (1, u8(4, 3))):
        with pytest.raises(ValueError):
            brq.mx_grouped_matmul(*ops[:i], bad, *ops[i + 1:])
    for bad in (dict(act="tanh"), dict(bias=f(6)), dict(bias=f(2, 5)), dict(mul=f(4, 5)), dict(residual=f(6)),
                dict(y=f(4, 5))):
        with pytest.raises(ValueError):
            brq.mx_grouped_matmul(*ops, **bad)

"""The edges of the paged attention with 16-bit queries and outputs, at the
lengths, windows, tables and values that test_gpu_kv.py takes float32 through,
and what is wrong in one query staying with it."""

import numpy as np
import pytest

from gpu_util import announce, to_dev, torch_dtype
from oracle import mx as X
from test_gpu_kv import EDGES, attend, build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,P,rot", [(64, 16, True), (64, 64, False), (128, 16, False), (128, 64, True), (256, 32, True)])
def test_lengths(D, P, rot, dtype):
    attend(EDGES, 4, 2, D, P, rot, dtype, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,hq", [(64, 6), (128, 6), (128, 24), (256, 3)])
@pytest.mark.parametrize("window", [1, 5, 16, 31, 32, 100, 1000])
def test_windows(window, D, hq, dtype):
    attend(EDGES, hq, 1, D, 16, False, dtype, window=window, seed=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_group_of_128(D, dtype):
    """All query heads over one key-value head: workgroups of 16 each."""
    attend([300, 0, 5, 1000], 128, 1, D, 32, True, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_and_peaked_softmax(scale, dtype):
    attend([400, 33], 8, 2, 128, 64, True, dtype, scale=scale, hot=True, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_split_sequence(D, dtype):
    attend([20011], 4, 1, D, 128, False, dtype, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_more_sequences_than_are_dealt_out(dtype):
    lens = np.random.default_rng(6).integers(0, 40, 4100)
    lens[[5, 4099]] = 700, 300
    attend(lens, 2, 1, 64, 16, True, dtype, seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pages_outside_the_cache_are_invisible(dtype):
    def edit(cache, ref, table):
        t = table.copy()
        t[0, 1], t[1, 0], t[1, 1], t[2, 0] = -1, cache.shape[0], -5, 2 ** 30
        return cache, ref, t
    out = attend([90, 40, 20], 4, 2, 128, 32, True, dtype, edit=edit, seed=7)
    assert not out[2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_key_or_value_reaches_only_who_sees_it(D, dtype):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention NaN key D={D} {dtype}")
    rng = np.random.default_rng(8)
    P, H, lens = 16, 2, [50, 50]
    cache, _, table, _, _, slots = build(rng, lens, H, D, P, False)
    q = torch.randn((2, 4, D), device="cuda").to(torch_dtype(dtype))
    ld, td = torch.tensor(lens, dtype=torch.int32, device="cuda"), to_dev(table, "i32")
    before = brq.paged_attention(None, q, cache, td, ld, P)
    assert torch.isfinite(before).all()
    e = D // 32 - 1
    for part in ("k", "v"):
        c = X.Cache.from_bytes(cache.cpu().numpy(), D, P)
        s = int(slots[7])  # token 7 of sequence 0, head 1
        (c.ks if part == "k" else c.vs)[s // P, 1, s % P, e] = 255
        bad = to_dev(c.to_bytes(), "u8")
        out = brq.paged_attention(None, q, bad, td, ld, P)
        assert torch.equal(out[1], before[1]) and torch.equal(out[0, :2], before[0, :2])
        nan = torch.isnan(out[0, 2:])
        assert nan.all() if part == "k" else (nan[:, 32 * e:].all() and not nan[:, :32 * e].any())
        assert torch.isfinite(brq.paged_attention(None, q, bad, td, ld, P, window=20)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,hq", [(64, 4), (128, 4), (128, 12), (256, 4)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_no_number_stays_alone(what, D, hq, dtype):
    """It makes its own head's output and lse NaN (a score is a sum with NaN or
    with infinities of either sign), nobody else's; one without a key to see
    comes to nothing."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention query {what} D={D} hq={hq} {dtype}")
    rng = np.random.default_rng(9)
    P, lens = 16, [50, 700, 0]
    cache, _, table, plan, _, _ = build(rng, lens, 1, D, P, True)
    q = torch.randn((3, hq, D), device="cuda").to(torch_dtype(dtype))
    ld, td = torch.tensor(lens, dtype=torch.int32, device="cuda"), to_dev(table, "i32")
    for p in (None, plan):
        lse0, lse = torch.empty((3, hq), device="cuda"), torch.empty((3, hq), device="cuda")
        before = brq.paged_attention(p, q, cache, td, ld, P, lse=lse0)
        bad = q.clone()
        bad[:, 1, D - 3] = what
        out = brq.paged_attention(p, bad, cache, td, ld, P, lse=lse)
        others = [h for h in range(hq) if h != 1]
        assert torch.equal(out[:, others], before[:, others]) and torch.equal(lse[:, others], lse0[:, others])
        assert torch.isnan(out[:2, 1]).all() and torch.isnan(lse[:2, 1]).all()
        assert not out[2].any() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_lengths_beyond_the_table_and_below_zero(dtype):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention lens out of range {dtype}")
    rng = np.random.default_rng(10)
    D, P = 64, 16
    cache, _, table, plan, _, _ = build(rng, [32, 32], 1, D, P, True)
    q = torch.randn((2, 2, D), device="cuda").to(torch_dtype(dtype))
    t = to_dev(np.ascontiguousarray(table[:, :2]), "i32")
    f = lambda lens: brq.paged_attention(plan, q, cache, t, torch.tensor(lens, dtype=torch.int32, device="cuda"), P)  # noqa: E731
    full = f([32, 32])
    assert torch.equal(f([2 ** 31 - 1, 33]), full)
    neg = f([-3, 32])
    assert not neg[0].any() and torch.equal(neg[1], full[1])

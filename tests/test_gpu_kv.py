"""GPU parity of the paged 4-bit key-value cache and of the attention that
reads it, against the oracle (oracle/mx.py).

The cache's bytes are compared bit for bit.  Attention's bound: a query enters
with 16 bits or more (as four 8-bit pieces, 2^-17 of its block's largest entry lost at
most; the losses of a block's entries have either sign, and their sum stays
under 2^-16 of the sum of magnitudes) after a float32 transform ((log2 D + 2)
2^-24 sqrt(D) of its largest entry, which the terms below cover with sqrt(D) to
spare); a score's D terms are summed in float32 (2^-23 each at
most); so a score is off by e = (2^-16 + 2 D 2^-23) times its sum of |q_i k_i|.
A probability then is off by a factor of exp(2 e), by 2^-17 of its pair and by
a few 2^-22 of its exponential; sums run over at most n / 32 + 96 additions of
2^-23.  The output adds its rounding."""

import numpy as np
import pytest

import synthetic as S
from gpu_util import announce, from_dev, lib_plan, to_dev, torch_dtype
from oracle import mx as X

pytestmark = pytest.mark.gpu

HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def rht(D):
    side = S.random_plan(np.random.default_rng(D), (2,) * (D.bit_length() - 1), "hadamard")
    return lib_plan(side), side.signs


def tokens(rng, n, H, D, dtype, gap=0):
    """A device [n, H, D] tensor (rows `gap` elements apart) and its float32 values."""
    import torch
    x = rng.standard_t(4, size=(n, H * D + gap)).astype(np.float32)
    t = torch.from_numpy(x).to(torch_dtype(dtype)).cuda()[:, :H * D].unflatten(1, (H, D))
    return t, t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,P,H,n,rot", [(64, 16, 3, 1, True), (64, 64, 1, 50, False), (128, 16, 8, 37, True),
                                         (128, 256, 2, 5, False), (256, 32, 5, 41, True)])
def test_append_and_read(D, P, H, n, rot, dtype):
    import butterfly_rotation_quantization_amd as brq
    announce(f"kv append/read D={D} P={P} H={H} n={n} rot={rot} {dtype}")
    rng = np.random.default_rng(D + P + n)
    pages = 6
    (k, kh), (v, vh) = tokens(rng, n, H, D, dtype, 16), tokens(rng, n, H, D, dtype, 48)
    plan, signs = rht(D) if rot else (None, None)
    slots = rng.permutation(pages * P)[:n].astype(np.int64)
    if n > 4:
        slots[1], slots[3] = -1, pages * P  # outside the cache: skipped
    raw = rng.integers(0, 256, (pages, H, P * (D + D // 16)), dtype=np.int64).astype(np.uint8)
    cache = to_dev(raw, "u8")
    brq.kv_append(plan, k, v, to_dev(slots, "i64"), cache, P)
    ref = X.Cache.from_bytes(raw, D, P)
    ref.append(kh, vh, slots, signs, rot)
    assert np.array_equal(cache.cpu().numpy(), ref.to_bytes())
    for un in ([None, plan] if rot else [None]):
        gk, gv = (from_dev(x) for x in brq.kv_read(un, cache, to_dev(slots, "i64"), D, P, out_dtype=torch_dtype(dtype)))
        K, V = ref.keys_values()
        for got, all_ in ((gk, K), (gv, V)):
            for i, s in enumerate(slots):
                if not 0 <= s < pages * P:
                    assert not got[i].any()
                    continue
                want = all_[s // P, :, s % P]
                if un is not None:
                    want = want @ X.hadamard64(D, signs)
                slack = 0.0 if un is None else (np.log2(D) + 2) * 2.0 ** -24 * np.sqrt(D) * np.abs(all_[s // P, :, s % P]).max()
                assert (np.abs(got[i] - want) <= slack + HALF_ULP[dtype] * np.abs(want)).all()


def build(rng, lens, H, D, P, rot, extra_pages=2, hot=False):
    """A cache holding lens[b] tokens of each sequence, its oracle, its table.
    Everything the sequences do not use is 0xFF: NaN scales and full codes."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    used = [(max(0, n) + P - 1) // P for n in lens]
    pages = sum(used) + extra_pages
    order = rng.permutation(pages)
    most = max(1, max(used)) + 1
    table = np.full((len(lens), most), 2 ** 31 - 1, dtype=np.int32)  # unused entries point nowhere
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        slots += [int(table[b, j // P]) * P + j % P for j in range(max(0, n))]
    slots = np.array(slots, dtype=np.int64)
    cache = torch.full((pages, H, P * (D + D // 16)), 255, dtype=torch.uint8, device="cuda")
    plan, signs = rht(D) if rot else (None, None)
    n = len(slots)
    k = rng.standard_normal((n, H, D)).astype(np.float32) * (4.0 if hot else 1.0)
    v = rng.standard_normal((n, H, D)).astype(np.float32) + 0.5
    if n:
        brq.kv_append(plan, to_dev(k, "f32"), to_dev(v, "f32"), to_dev(slots, "i64"), cache, P)
    M = X.hadamard64(D, signs) if rot else None
    return cache, X.Cache.from_bytes(cache.cpu().numpy(), D, P), table, plan, M, slots


def check(got, lse, want, wlse, slack, lens, D, dtype, scale_terms=True):
    spread, terms = slack
    e = (2.0 ** -16 + 2 * D * 2.0 ** -23) * terms  # [B, hq]
    rel = 2 * e + 2.0 ** -16 + (np.maximum(0, np.asarray(lens)) / 32 + 96)[:, None] * 2.0 ** -23
    bound = 2 * rel[..., None] * spread + HALF_ULP[dtype] * np.abs(want) + 2.0 ** -25
    over = np.abs(got - want) > bound
    assert not over.any(), (f"{int(over.sum())} outputs beyond the bound, first {np.argwhere(over)[:3].tolist()}, "
                            f"largest error {np.abs(got - want).max():.3g}")
    fine = np.isfinite(wlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(wlse))
    assert (np.abs(lse[fine] - wlse[fine]) <= (2 * rel + 2.0 ** -22 * (1 + np.abs(np.where(fine, wlse, 0))))[fine]).all()


def attend(lens, hq, H, D, P, rot, dtype, window=0, scale=None, hot=False, seed=0, edit=None):
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention lens={list(lens)[:6]} hq={hq} H={H} D={D} P={P} rot={rot} {dtype} window={window}")
    rng = np.random.default_rng(seed + D + P + hq)
    cache, ref, table, plan, M, _ = build(rng, lens, H, D, P, rot, hot=hot)
    if edit:
        cache, ref, table = edit(cache, ref, table)
    B = len(lens)
    q, qh = tokens(rng, B, hq, D, dtype, 32)
    ld = torch.tensor(np.asarray(lens, dtype=np.int32), device="cuda")
    lse = torch.full((B, hq), 7.0, device="cuda")
    out = brq.paged_attention(plan, q, cache, to_dev(table, "i32"), ld, P, scale=scale, window=window, lse=lse)
    again = brq.paged_attention(plan, q, cache, to_dev(table, "i32"), ld, P, scale=scale, window=window)
    assert torch.equal(out.view(torch.int16 if dtype != "f32" else torch.int32),
                       again.view(torch.int16 if dtype != "f32" else torch.int32)), "a second call differs"
    want, wlse, slack = X.attention(qh.astype(np.float64), ref, table, lens, D ** -0.5 if scale is None else scale,
                                    window, M)
    check(from_dev(out), from_dev(lse), want, wlse, slack, lens, D, dtype)
    return out


# lengths around the 16 and 32 keys of a tile, the 128 of a workgroup, a page
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P,rot", [(16, True), (64, False)])
def test_lengths(D, P, rot):
    attend(EDGES, 4, 2, D, P, rot, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,H", [(1, 1), (8, 8), (9, 1), (16, 1), (40, 2), (20, 1), (33, 1), (24, 8)])
def test_head_groups(hq, H, dtype):
    attend([77, 0, 300, 1], hq, H, 128, 32, True, dtype)


@pytest.mark.parametrize("D", [64, 256])
def test_wide_groups(D):
    attend([130, 3], 48, 2, D, 16, True, "bf16")


@pytest.mark.parametrize("window", [1, 5, 16, 31, 32, 100, 1000])
def test_windows(window):
    attend(EDGES, 6, 2, 128, 16, False, "f32", window=window)


@pytest.mark.parametrize("D,hq,rot", [(64, 8, True), (128, 8, True), (128, 40, False), (256, 3, True)])
def test_float32_keeps_float32(D, hq, rot):
    """Scores of a few units are off by some 2^-21 in float32 (products of 24
    bits, sums of D terms of either sign, one exponential), and the output, a
    mean of values around 0.5, by no more than twice that in the mean: 2^-18 of
    its norm leaves a factor of four.  Probabilities or queries of 16 bits
    would be at 2^-17."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention float32 D={D} hq={hq} rot={rot}")
    rng = np.random.default_rng(D + hq)
    lens = [150, 700]
    cache, ref, table, plan, M, _ = build(rng, lens, 1, D, 64, rot)
    q = torch.from_numpy(rng.standard_normal((2, hq, D)).astype(np.float32)).cuda()
    out = brq.paged_attention(plan, q, cache, to_dev(table, "i32"), torch.tensor(lens, dtype=torch.int32).cuda(), 64)
    want, _, _ = X.attention(q.cpu().numpy().astype(np.float64), ref, table, lens, D ** -0.5, 0, M)
    assert np.linalg.norm(from_dev(out) - want) < 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_small_entries_of_a_query_count(D, dtype):
    """One key of ones, so that lse is the sum of the query: every entry counts,
    however far below the largest of its block it lies, to 2^-17 of that one
    (float32: 2^-22), which the additions' 2^-22 of the sum, log and exponential
    stay within too."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce(f"attention of small query entries D={D} {dtype}")
    cache = brq.kv_cache(1, 1, D, 16)
    ones = torch.ones((1, 1, D), device="cuda")
    brq.kv_append(None, ones, ones, torch.zeros(1, dtype=torch.int64, device="cuda"), cache, 16)
    q = torch.zeros((1, 24, D), device="cuda")
    q[0, :, 3] = 1.0
    q[0, :, 5] = -(2.0 ** -torch.arange(24, device="cuda"))
    q = q.to(torch_dtype(dtype))
    lse = torch.empty((1, 24), device="cuda")
    brq.paged_attention(None, q, cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                        torch.ones(1, dtype=torch.int32, device="cuda"), 16, scale=1.0, lse=lse)
    off = (lse.double() - q.double().sum(-1)).abs().max().item()
    assert off <= (2.0 ** -21 if dtype == "f32" else 2.0 ** -17 + 2.0 ** -21), off


def test_long_and_ragged():
    attend([20011, 1, 4099, 0, 777], 8, 2, 128, 64, True, "bf16")


def test_single_long_sequence_is_split():
    attend([33333], 4, 1, 128, 128, False, "f32")


def test_many_sequences():
    rng = np.random.default_rng(0)
    attend(rng.integers(0, 120, 300), 8, 4, 64, 16, True, "f16")


def test_more_sequences_than_are_dealt_out():
    """Above 4096 sequences each group of heads has a workgroup of its own."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, 4100)
    lens[77] = 700
    attend(lens, 2, 1, 64, 16, True, "f32")


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_and_peaked_softmax(scale):
    attend([400, 33], 8, 2, 128, 64, True, "f32", scale=scale, hot=True)


def test_pages_outside_the_cache_are_invisible():
    """A sequence whose table names pages that do not exist: their tokens drop
    out; with none left the output is zero."""
    def edit(cache, ref, table):
        t = table.copy()
        t[0, 1], t[1, 0], t[1, 1], t[2, 0] = -1, cache.shape[0], -5, 2 ** 30
        return cache, ref, t
    out = attend([90, 40, 20], 4, 2, 128, 32, True, "f32", edit=edit)
    assert not out[2].any()


def test_a_cache_without_pages():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("attention over no pages")
    cache = brq.kv_cache(0, 2, 128, 32)
    table, lens = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.tensor([40, 0, 1], dtype=torch.int32).cuda()
    lse = torch.zeros((3, 4), device="cuda")
    out = brq.paged_attention(None, torch.randn((3, 4, 128), device="cuda"), cache, table, lens, 32, lse=lse)
    assert not out.any() and torch.isneginf(lse).all()


def test_a_nan_key_or_value_reaches_only_who_sees_it():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("attention NaN key")
    rng = np.random.default_rng(4)
    D, P, H = 128, 16, 2
    lens = [50, 50]
    cache, ref, table, _, _, slots = build(rng, lens, H, D, P, False)
    q = torch.randn((2, 4, D), device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = brq.paged_attention(None, q, cache, to_dev(table, "i32"), ld, P)
    assert torch.isfinite(before).all()
    for part in ("k", "v"):
        c = X.Cache.from_bytes(cache.cpu().numpy(), D, P)
        s = int(slots[7])  # token 7 of sequence 0, head 1
        (c.ks if part == "k" else c.vs)[s // P, 1, s % P, 2] = 255
        out = brq.paged_attention(None, q, to_dev(c.to_bytes(), "u8"), to_dev(table, "i32"), ld, P)
        assert torch.equal(out[1], before[1]) and torch.equal(out[0, :2], before[0, :2])
        nan = torch.isnan(out[0, 2:])
        assert nan.all() if part == "k" else (nan[:, 64:96].all() and not nan[:, :64].any() and not nan[:, 96:].any())
        # out of the window it is not seen
        w = brq.paged_attention(None, q, to_dev(c.to_bytes(), "u8"), to_dev(table, "i32"), ld, P, window=20)
        assert torch.isfinite(w).all()


def test_lengths_beyond_the_table_and_below_zero():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("attention lens out of range")
    rng = np.random.default_rng(6)
    D, P = 64, 16
    cache, ref, table, plan, M, _ = build(rng, [32, 32], 1, D, P, True)
    q = torch.randn((2, 2, D), device="cuda")
    t = to_dev(np.ascontiguousarray(table[:, :2]), "i32")
    f = lambda lens: brq.paged_attention(plan, q, cache, t, torch.tensor(lens, dtype=torch.int32, device="cuda"), P)  # noqa: E731
    full = f([32, 32])
    assert torch.equal(f([2 ** 31 - 1, 33]), full)
    neg = f([-3, 32])
    assert not neg[0].any() and torch.equal(neg[1], full[1])


def test_output_may_be_the_query():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("attention in place")
    rng = np.random.default_rng(7)
    for B, n in ((1, 3000), (200, 40)):  # with and without a split
        cache, _, table, plan, _, _ = build(rng, [n] * B, 4, 128, 32, True)
        q = torch.randn((B, 8, 128), device="cuda").to(torch.bfloat16)
        ld = torch.full((B,), n, dtype=torch.int32, device="cuda")
        want = brq.paged_attention(plan, q, cache, to_dev(table, "i32"), ld, 32)
        brq.paged_attention(plan, q, cache, to_dev(table, "i32"), ld, 32, out=q)
        assert torch.equal(q, want)


def test_cache_beyond_32_bit_offsets():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("cache of 4.7 GB")
    H, D, P = 8, 128, 64
    pages = 68000
    rng = np.random.default_rng(8)
    cache = brq.kv_cache(pages, H, D, P)
    n = 70
    (k, kh), (v, vh) = tokens(rng, n, H, D, "bf16"), tokens(rng, n, H, D, "bf16")
    table = np.array([[pages - 1, pages - 3]], dtype=np.int32)
    slots = np.array([int(table[0, j // P]) * P + j % P for j in range(n)], dtype=np.int64)
    brq.kv_append(None, k, v, to_dev(slots, "i64"), cache, P)
    last = cache[-3:].cpu().numpy()
    assert not cache[:-3].any()
    ref = X.Cache(3, H, D, P)
    ref.append(kh, vh, slots - (pages - 3) * P)
    assert np.array_equal(last, ref.to_bytes())
    gk, _ = brq.kv_read(None, cache, to_dev(slots, "i64"), D, P)
    assert np.array_equal(from_dev(gk)[0], ref.keys_values()[0][2, :, 0])
    q, qh = tokens(rng, 1, 16, D, "f32")
    lse = torch.empty((1, 16), device="cuda")
    out = brq.paged_attention(None, q, cache, to_dev(table, "i32"), torch.tensor([n], dtype=torch.int32, device="cuda"),
                              P, lse=lse)
    want, wlse, slack = X.attention(qh.astype(np.float64), ref, table - (pages - 3), [n], D ** -0.5)
    check(from_dev(out), from_dev(lse), want, wlse, slack, [n], D, "f32")


def test_a_captured_step_follows_growing_sequences():
    """Append and attention captured once and replayed while lengths and slots
    change on the device, against eager calls on a copy of the cache."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("attention graph")
    rng = np.random.default_rng(9)
    H, D, P, B = 2, 128, 16, 3
    cache, _, table, plan, _, _ = build(rng, [40, 5, 90], H, D, P, True, extra_pages=9)
    free = [p for p in range(cache.shape[0]) if p not in table]
    table = np.concatenate([table, np.zeros((B, 3), np.int32)], axis=1)
    lens = np.array([40, 5, 90])
    for b in range(B):  # two more pages for each sequence
        u = (lens[b] + P - 1) // P
        table[b, u:u + 2] = free[2 * b:2 * b + 2]
    td = to_dev(np.ascontiguousarray(table), "i32")
    k, v = (torch.randn((B, H, D), device="cuda") for _ in range(2))
    q = torch.randn((B, 8, D), device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    ld = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = brq.paged_attention_workspace(B, 8, H, D)
    other = cache.clone()

    def set_step(i):
        n = lens + i
        slots.copy_(torch.tensor([int(table[b, n[b] // P]) * P + n[b] % P for b in range(B)]))
        ld.copy_(torch.tensor(n + 1, dtype=torch.int32))
        k.normal_(), v.normal_(), q.normal_()

    def step():
        brq.kv_append(plan, k, v, slots, cache, P)
        brq.paged_attention(plan, q, cache, td, ld, P, out=out, ws=ws)
    set_step(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    brq.kv_append(plan, k, v, slots, other, P)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for i in range(1, 20):
        set_step(i)
        brq.kv_append(plan, k, v, slots, other, P)
        want = brq.paged_attention(plan, q, other, td, ld, P)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, other) and torch.equal(out, want), f"replay {i} differs"


def test_binding_refuses_other_layouts():
    import butterfly_rotation_quantization_amd as brq
    import torch
    cache = brq.kv_cache(2, 2, 64, 16)
    q = torch.zeros((1, 4, 64), device="cuda")
    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    ln = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.zeros((3, 2, 64), device="cuda")
    sl = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        brq.paged_attention(None, q, cache, t.long(), ln, 16)
    with pytest.raises(ValueError):
        brq.paged_attention(None, q, cache, t, ln, 32)
    with pytest.raises(ValueError):
        brq.paged_attention(None, q, cache, t, ln, 16, out=q.half())
    with pytest.raises(ValueError):
        brq.kv_append(None, k, k, sl.int(), cache, 16)
    with pytest.raises(ValueError):
        brq.kv_append(None, k, k.half(), sl, cache, 16)
    with pytest.raises(ValueError):
        brq.kv_read(None, cache, sl, 128, 16)
    with pytest.raises(brq.BrqError):
        brq.kv_cache(2, 2, 80, 16)

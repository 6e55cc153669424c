"""Tokens and pages of the paged 4-bit cache moved, shared, taken and given
back, against the oracle (oracle/mx.py): bytes, tables and counts are compared
one for one."""

import numpy as np
import pytest

from gpu_util import announce, to_dev
from oracle import mx as X

pytestmark = pytest.mark.gpu


def full_cache(rng, pages, H, D, P):
    """A cache of arbitrary bytes, on the device and in the oracle's layout."""
    raw = rng.integers(0, 256, (pages, H, P * (D + D // 16)), dtype=np.int64).astype(np.uint8)
    return to_dev(raw, "u8"), X.Cache.from_bytes(raw, D, P)


def same(cache, ref):
    return np.array_equal(cache.cpu().numpy(), ref.to_bytes())


@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 64, 8), (128, 16, 1), (256, 32, 5), (64, 1024, 2)])
@pytest.mark.parametrize("n", [1, 5, 40, 700, 3000])
def test_move(D, P, H, n):
    import butterfly_rotation_quantization_amd as brq
    announce(f"kv move D={D} P={P} H={H} n={n}")
    rng = np.random.default_rng(D + P + n)
    pages = max(4, (2 * n + P - 1) // P)
    cache, ref = full_cache(rng, pages, H, D, P)
    src, dst = rng.integers(0, pages * P, n), rng.permutation(pages * P)[:n]  # tokens copied twice, overwritten, moved on
    if n > 4:
        src[1], dst[2], src[3], dst[4] = -1, -1, pages * P, 2 ** 40
    brq.kv_move(cache, to_dev(src.astype(np.int64), "i64"), to_dev(dst.astype(np.int64), "i64"), D, P)
    X.move(ref, src, dst)
    assert same(cache, ref)


@pytest.mark.parametrize("n", [64, 512, 513, 2000])
def test_move_reads_all_before_it_writes(n):
    """A rotation by one place, a reversal, and every token one place down: each overlaps with itself everywhere."""
    import butterfly_rotation_quantization_amd as brq
    announce(f"kv move overlapping n={n}")
    rng = np.random.default_rng(n)
    D, P, H = 128, 32, 4
    cache, ref = full_cache(rng, (n + P) // P + 1, H, D, P)
    i = np.arange(n, dtype=np.int64)
    for src, dst in ((i, (i + 1) % n), (i, i[::-1].copy()), (i + 1, i)):
        brq.kv_move(cache, to_dev(src, "i64"), to_dev(dst, "i64"), D, P)
        X.move(ref, src, dst)
        assert same(cache, ref)


def test_moved_tokens_read_back():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("kv move and read")
    P, D, H = 16, 128, 2
    cache = brq.kv_cache(8, H, D, P)
    k, v = (torch.randn((6, H, D), device="cuda") for _ in range(2))
    slots = torch.tensor([3, 17, 40, 41, 90, 127], device="cuda")
    brq.kv_append(None, k, v, slots, cache, P)
    before = brq.kv_read(None, cache, slots, D, P)
    to = torch.tensor([17, 3, 64, 65, 66, 0], device="cuda")
    brq.kv_move(cache, slots, to, D, P)
    after = brq.kv_read(None, cache, to, D, P)
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def pool(rng, lens, P, W, pages):
    """A table of distinct pages for sequences of these lengths, and how many rows hold each page."""
    order = list(rng.permutation(pages))
    table, refs = np.full((len(lens), W), -1, np.int32), np.zeros(pages, np.int32)
    for b, n in enumerate(lens):
        for c in range((max(0, n) + P - 1) // P):
            table[b, c] = order.pop()
            refs[table[b, c]] += 1
    return table, refs


@pytest.mark.parametrize("B,W,F", [(1, 1, 1), (3, 5, 7), (4, 300, 130), (2, 0, 3), (0, 4, 2)])
def test_fork(B, W, F):
    import butterfly_rotation_quantization_amd as brq
    announce(f"kv fork B={B} W={W} F={F}")
    rng = np.random.default_rng(B + W + F)
    P, pages = 16, max(1, B * W)
    lens = rng.integers(0, W * P + 1, B).astype(np.int32)
    table, refs = pool(rng, lens, P, W, pages)
    if B and W > 2:
        table[0, W - 1], table[-1, 0] = pages + 3, -2 ** 31  # no pages
    parents = rng.integers(-1, B + 1, F).astype(np.int32)
    dev = [to_dev(x, "i32") for x in (table, lens, parents, refs)]
    got = brq.kv_fork(*dev)
    want = X.fork(table, lens, parents, refs)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))
    assert np.array_equal(dev[3].cpu().numpy(), refs) and np.array_equal(dev[0].cpu().numpy(), table)


def run_reserve(cache, ref, table, lens, refs, N, D, P, slots=None, ws=None):
    import butterfly_rotation_quantization_amd as brq
    t, n, r = (to_dev(np.ascontiguousarray(x, dtype=np.int32), "i32") for x in (table, lens, refs))
    got = brq.kv_reserve(cache, t, n, r, N, D, P, slots=slots, ws=ws)
    want = X.reserve(ref, table, lens, refs, N)
    assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert same(cache, ref)
    return want


@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 64, 8), (256, 32, 1), (128, 256, 2)])
@pytest.mark.parametrize("N", [1, 5, 33, 300])
def test_reserve(D, P, H, N):
    """Sequences that hold their pages alone, that share them twice and three times, of every place in a page."""
    announce(f"kv reserve D={D} P={P} H={H} N={N}")
    rng = np.random.default_rng(D + P + N)
    W = (3 * P + N) // P + 1
    lens = np.array([0, 1, 15, 16, 17, P - 1, P, P + 1, 3 * P, -1, -7])
    pages = 14 * W + 4
    cache, ref = full_cache(rng, pages, H, D, P)
    table, refs = pool(rng, lens, P, W, pages)
    parents = np.array([1, 4, 5, 7, 7, 8, 2, 0, 9])
    kids, klens = X.fork(table, lens, parents, refs)
    run_reserve(cache, ref, np.concatenate((table, kids)), np.concatenate((lens, klens)), refs, N, D, P)


def test_reserve_when_every_owner_asks():
    """All rows that hold a page ask at once: each gets a copy, the page is free afterwards."""
    announce("kv reserve, every owner")
    rng = np.random.default_rng(5)
    P, D, H, W = 16, 64, 2, 3
    cache, ref = full_cache(rng, 12, H, D, P)
    table, refs = pool(rng, [20], P, W, 12)
    kids, lens = X.fork(table, [20], [0, 0, 0], refs)
    X.free(table, refs, [0])
    old = kids[0, 1]
    run_reserve(cache, ref, kids, lens, refs, 2, D, P)
    assert refs[old] == 0 and refs[kids[0, 0]] == 3


@pytest.mark.parametrize("left", [0, 1, 3, 6])
def test_reserve_from_a_pool_that_runs_out(left):
    """The first sequences get what is left; the others' entries stay, their slots are -1."""
    announce(f"kv reserve, {left} pages left")
    rng = np.random.default_rng(left)
    P, D, H, W = 16, 64, 1, 4
    lens = [5, 16, 20, 40, 16]
    table, refs = pool(rng, lens, P, W, 9)
    assert (refs == 0).sum() == 9 - sum((n + P - 1) // P for n in lens)
    kids, klens = X.fork(table, lens, [0, 2], refs)
    for p in np.flatnonzero(refs == 0)[left:]:
        refs[p] = 1
    cache, ref = full_cache(rng, 9, H, D, P)
    slots = run_reserve(cache, ref, np.concatenate((table, kids)), np.concatenate((lens, klens)), refs, 20, D, P)
    assert (slots == -1).any()


def test_reserve_beyond_the_table():
    announce("kv reserve beyond the table")
    rng = np.random.default_rng(1)
    P, D, H, W = 16, 64, 1, 2
    cache, ref = full_cache(rng, 20, H, D, P)
    lens = np.array([30, 32, 31, 2 ** 31 - 1, 0, 1000])
    table, refs = pool(rng, [30, 32, 31, 32, 0, 32], P, W, 20)
    run_reserve(cache, ref, table, lens, refs, 40, D, P)


@pytest.mark.parametrize("B,pages", [(1500, 4000), (3000, 70000)])
def test_reserve_for_many(B, pages):
    """More entries and pages than the deciding workgroup has threads."""
    announce(f"kv reserve B={B} pages={pages}")
    rng = np.random.default_rng(B)
    P, D, H, W = 16, 64, 1, 3
    lens = rng.integers(-1, 2 * P, B)
    refs = np.where(rng.random(pages) < 0.97, 1, 0).astype(np.int32)
    refs[-B:] = 0
    table = np.full((B, W), -1, np.int32)
    held = np.flatnonzero(refs[:-B] == 1)
    table[:, 0] = rng.permutation(held)[:B] if len(held) >= B else rng.choice(held, B)
    refs[:] = np.where(refs > 0, 1, 0)
    for p in table[:, 0]:
        refs[p] = 0
    for p in table[:, 0]:
        refs[p] += 1
    cache, ref = full_cache(rng, pages, H, D, P)
    run_reserve(cache, ref, table, lens, refs, 20, D, P)


def test_free():
    import butterfly_rotation_quantization_amd as brq
    announce("kv free")
    rng = np.random.default_rng(2)
    P, W, pages = 16, 40, 300
    lens = rng.integers(0, W * P, 6)
    table, refs = pool(rng, lens, P, W, pages)
    kids, _ = X.fork(table, lens, [0, 0, 3], refs)
    table = np.concatenate((table, kids))
    table[5, W - 1] = pages + 1  # no page: cleared, not counted
    for rows in (np.array([0, 7, 0, -1, 9, 100], np.int32), None, None):  # the same row twice, rows that are none; all; again
        t, r = to_dev(table, "i32"), to_dev(refs, "i32")
        brq.kv_free(t, r, None if rows is None else to_dev(rows, "i32"))
        X.free(table, refs, range(len(table)) if rows is None else rows)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert not refs.any() and (table == -1).all()


def test_a_captured_loop_of_samples():
    """Forks, reservations, appends, moves and frees in one graph, replayed while
    lengths change on the device, against the oracle."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("kv pages graph")
    rng = np.random.default_rng(3)
    P, D, H, W, pages, N = 16, 128, 2, 6, 60, 5
    lens = np.array([20, 33, 16], np.int32)
    cache, ref = full_cache(rng, pages, H, D, P)
    table, refs = pool(rng, lens, P, W, pages)
    parents = np.array([0, 1, 1, 2, 0], np.int32)
    t, n, r, par = (to_dev(x, "i32") for x in (table, lens, refs, parents))
    kt, kn = torch.zeros((5, W), dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    slots = torch.zeros((5, N), dtype=torch.int64, device="cuda")
    k, v = (torch.randn((5 * N, H, D), device="cuda") for _ in range(2))
    ws = brq.kv_reserve_workspace(5, N, P, pages), brq.kv_move_workspace(10, H, D)

    def step():
        brq.kv_fork(t, n, par, r, kt, kn)
        brq.kv_reserve(cache, kt, kn, r, N, D, P, slots=slots, ws=ws[0])
        brq.kv_append(None, k, v, slots.view(-1), cache, P)
        brq.kv_move(cache, slots[:, 3:].contiguous().view(-1), slots[:, 1:3].contiguous().view(-1), D, P, ws=ws[1])
        brq.kv_free(kt, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = cache.clone()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    cache.copy_(saved)
    torch.cuda.synchronize()
    for i in range(5):
        m = (lens - i).astype(np.int32)
        n.copy_(torch.from_numpy(m))
        for w in ws:
            if w is not None:
                w.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        kids, klens = X.fork(table, m, parents, refs)
        want = X.reserve(ref, kids, klens, refs, N)
        assert np.array_equal(slots.cpu().numpy(), want), i
        ref.append(k.cpu().numpy(), v.cpu().numpy(), want.reshape(-1))
        X.move(ref, want[:, 3:].reshape(-1), want[:, 1:3].reshape(-1))
        X.free(kids, refs, range(5))
        assert same(cache, ref) and np.array_equal(r.cpu().numpy(), refs), i
        assert (kt == -1).all()


def test_pages_nothing_to_do_and_refusals():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("kv pages refusals")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")  # noqa: E731
    cache = brq.kv_cache(4, 2, 64, 16)
    brq.kv_move(cache, i64(0), i64(0), 64, 16)
    assert brq.kv_fork(i32(2, 3), i32(2), i32(0), i32(4))[0].shape == (0, 3)
    assert brq.kv_reserve(cache, i32(0, 3), i32(0), i32(4), 2, 64, 16).shape == (0, 2)
    assert brq.kv_reserve(cache, i32(2, 3), i32(2), i32(4), 0, 64, 16).shape == (2, 0)
    brq.kv_free(i32(0, 3), i32(4)), brq.kv_free(i32(2, 0), i32(4)), brq.kv_free(i32(2, 3), i32(4), i32(0))
    assert (brq.kv_reserve(brq.kv_cache(0, 2, 64, 16), i32(2, 3), i32(2), i32(0), 2, 64, 16) == -1).all()
    bad = [lambda: brq.kv_move(cache, i32(3), i64(3), 64, 16), lambda: brq.kv_move(cache, i64(3), i64(2), 64, 16),
           lambda: brq.kv_move(cache, i64(3), i64(3), 128, 16), lambda: brq.kv_move(cache, i64(3).cpu(), i64(3), 64, 16),
           lambda: brq.kv_fork(i32(6), i32(2), i32(1), i32(4)), lambda: brq.kv_fork(i32(2, 3), i32(3), i32(1), i32(4)),
           lambda: brq.kv_fork(i32(2, 3), i32(2), i64(1), i32(4)),
           lambda: brq.kv_fork(i32(2, 3), i32(2), i32(1), i32(4), out_table=i32(2, 3)),
           lambda: brq.kv_reserve(cache, i32(2, 3), i32(2), i32(5), 2, 64, 16),
           lambda: brq.kv_reserve(cache, i32(2, 3), i32(2), i32(4), 2, 64, 32),
           lambda: brq.kv_reserve(cache, i32(3, 2).t(), i32(2), i32(4), 2, 64, 16),
           lambda: brq.kv_reserve(cache, i32(2, 3), i32(2), i32(4), 2, 64, 16, slots=i64(2, 3)),
           lambda: brq.kv_free(i32(6), i32(4)), lambda: brq.kv_free(i32(2, 3), i64(4)),
           lambda: brq.kv_free(i32(2, 3), i32(4), i64(1))]
    for f in bad:
        with pytest.raises(ValueError):
            f()

"""CPU checks of the tree attention and of the cache's moves, forks,
reservations and frees: the dry run of their launches, every refusal with fake device
addresses that are never dereferenced, and the binding with tensors that only
say where they are."""

import numpy as np
import pytest
import torch

import butterfly_rotation_quantization_amd as brq
import synthetic as S
from test_host_dryrun import DPlan, _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import ALIGNMENT, CACHE, INVALID, LENS, SLOTS, TABLE, UNSUPPORTED, WORKSPACE, WS, X, Y, rht
from test_host_mx_binding import At, library, u8  # noqa: F401

MASK, REFS, OTHER, MORE = 0x1000000000, 0x1100000000, 0x1200000000, 0x1300000000


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,N,hq,H,P,ldt", [(1, 7, 32, 8, 64, 20), (32, 8, 64, 8, 32, 512), (4, 64, 64, 8, 128, 300),
                                            (3, 1, 5, 1, 16, 9), (64, 3, 24, 24, 1024, 4), (2, 5, 9, 1, 16, 0),
                                            (4097, 4, 8, 2, 16, 6), (1, 11, 16, 1, 256, 1 << 20)])
def test_tree_walk(dl, D, B, N, hq, H, P, ldt):  # noqa: F811
    plan = rht(dl, D)
    nb = dl.brq_tree_attention_workspace_bytes(B, N, hq, H, D)
    assert (nb == 0) == (B > 4096)
    for h in (None, plan.h):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_tree_attention(h, X, hq * D, 1, CACHE, 1000, TABLE, ldt, LENS, MASK, B, N, hq, H, D, P, 0.1, 0,
                                      Y, hq * D, None, WS if nb else None, nb, None), f"tree {B}x{N}")
        assert dl.brq_dryrun_launches() == 1


def test_tree_refusals(dl):  # noqa: F811
    def f(h=None, q=X, ldq=1024, t=1, c=CACHE, pages=9, table=TABLE, ldt=5, lens=LENS, mask=MASK, B=3, N=4, hq=8, H=2,
          D=128, P=64, scale=0.1, window=0, out=Y, ldo=1024, lse=None, ws=WS, less=0):
        nb = dl.brq_tree_attention_workspace_bytes(B, N, hq, H, D) - less
        return dl.brq_tree_attention(h, q, ldq, t, c, pages, table, ldt, lens, mask, B, N, hq, H, D, P, scale, window,
                                     out, ldo, lse, ws, max(nb, 0), None)
    assert f() == 0 and f(B=0, q=None) == 0 and f(N=0, mask=None) == 0 and f(pages=0, c=None) == 0 and f(ldt=0, table=None) == 0
    for bad in (dict(t=4), dict(B=-1), dict(N=-1), dict(H=0), dict(hq=0), dict(hq=7), dict(pages=-1), dict(ldt=-1),
                dict(window=-1), dict(scale=float("inf")), dict(ldq=1016), dict(ldo=1016), dict(q=None), dict(out=None),
                dict(lens=None), dict(mask=None), dict(table=None), dict(c=None)):
        assert f(**bad) == INVALID, bad
    p64, dense = rht(dl, 64), DPlan(dl, S.random_plan(np.random.default_rng(1), (8, 16), "per_group"))
    for bad in (dict(D=96), dict(P=48), dict(P=8), dict(N=65), dict(h=p64.h), dict(h=dense.h), dict(B=1 << 20, N=2),
                dict(B=(1 << 24) // 32)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=X + 8), dict(ldq=1028), dict(out=Y + 8), dict(c=CACHE + 8), dict(table=TABLE + 2),
                dict(lens=LENS + 1), dict(mask=MASK + 4), dict(lse=Y + 2), dict(ws=WS + 8)):
        assert f(**bad) == ALIGNMENT, bad
    assert f(ws=None) == WORKSPACE and f(less=1) == WORKSPACE
    for bad in ((0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 65, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 1, 2, 128), (1, 1, 8, 2, 96)):
        assert dl.brq_tree_attention_workspace_bytes(*bad) == 0
    assert dl.brq_last_error()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 64, 1024])
def test_pages_walk(dl, D, P):  # noqa: F811
    for n in (1, 512, 513, 100001):
        nb = dl.brq_kv_move_workspace_bytes(n, 3, D)
        assert (nb == 0) == (n <= 512)
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_kv_move(CACHE, SLOTS, OTHER, n, 3, D, P, 11, WS if nb else None, nb, None), "move")
        assert dl.brq_dryrun_launches() == 1
    for B, W, N in ((1, 1, 1), (7, 40, P), (300, 9, 3 * P + 5), (2, 0, 4)):
        nb = dl.brq_kv_reserve_workspace_bytes(B, N, P, 500)
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_kv_reserve(CACHE, TABLE, LENS, B, W, REFS, 500, N, 3, D, P, SLOTS, WS, nb, None), "reserve")
        _ok(dl, dl.brq_kv_fork(TABLE, LENS, B, W, OTHER, 9, REFS, 500, MORE, MORE + 4096, None), "fork")
        _ok(dl, dl.brq_kv_free(TABLE, B, W, REFS, 500, OTHER, 9, None), "free")
        assert dl.brq_dryrun_launches() == (3 if W else 2)


def test_pages_refusals(dl):  # noqa: F811
    def move(c=CACHE, s=SLOTS, d=OTHER, n=1000, H=8, D=128, P=64, pages=9, ws=WS, less=0):
        nb = dl.brq_kv_move_workspace_bytes(n, H, D) - less
        return dl.brq_kv_move(c, s, d, n, H, D, P, pages, ws, max(nb, 0), None)
    assert move() == 0 and move(n=0, s=None) == 0 and move(pages=0, c=None) == 0 and move(n=5, ws=None) == 0
    for bad in (dict(n=-1), dict(H=0), dict(pages=-1), dict(c=None), dict(s=None), dict(d=None)):
        assert move(**bad) == INVALID, bad
    assert move(D=80) == UNSUPPORTED and move(P=24) == UNSUPPORTED and move(n=(1 << 24) + 1) == UNSUPPORTED
    assert move(c=CACHE + 8) == ALIGNMENT and move(s=SLOTS + 4) == ALIGNMENT and move(d=OTHER + 1) == ALIGNMENT
    assert move(ws=None) == WORKSPACE and move(less=1) == WORKSPACE and move(ws=WS + 8) == ALIGNMENT

    def fork(t=TABLE, n=LENS, B=3, W=5, p=OTHER, F=4, r=REFS, pages=9, ot=MORE, on=Y):
        return dl.brq_kv_fork(t, n, B, W, p, F, r, pages, ot, on, None)
    assert fork() == 0 and fork(F=0, p=None) == 0 and fork(B=0, t=None, n=None) == 0 and fork(W=0, t=None, ot=None) == 0
    assert fork(pages=0, r=None) == 0
    for bad in (dict(B=-1), dict(W=-1), dict(F=-1), dict(pages=-1), dict(t=None), dict(n=None), dict(p=None), dict(r=None),
                dict(ot=None), dict(on=None)):
        assert fork(**bad) == INVALID, bad
    assert fork(B=1 << 20, W=1 << 11) == UNSUPPORTED and fork(F=1 << 31, W=0) == UNSUPPORTED and fork(pages=1 << 31) == UNSUPPORTED
    for k in ("t", "n", "p", "r", "ot", "on"):
        assert fork(**{k: TABLE + 2}) == ALIGNMENT, k

    def reserve(c=CACHE, t=TABLE, n=LENS, B=3, W=5, r=REFS, pages=9, N=4, H=8, D=128, P=64, s=SLOTS, ws=WS, less=0):
        nb = dl.brq_kv_reserve_workspace_bytes(B, N, P, pages) - less
        return dl.brq_kv_reserve(c, t, n, B, W, r, pages, N, H, D, P, s, ws, max(nb, 0), None)
    assert reserve() == 0 and reserve(B=0, n=None) == 0 and reserve(N=0, s=None) == 0 and reserve(W=0, t=None) == 0
    assert reserve(pages=0, c=None, r=None) == 0
    for bad in (dict(B=-1), dict(W=-1), dict(N=-1), dict(H=0), dict(pages=-1), dict(c=None), dict(t=None), dict(n=None),
                dict(r=None), dict(s=None)):
        assert reserve(**bad) == INVALID, bad
    for bad in (dict(D=80), dict(P=20), dict(H=65536), dict(B=1 << 24), dict(B=1 << 20, W=1 << 11), dict(pages=1 << 31),
                dict(B=1 << 20, N=1 << 20)):
        assert reserve(**bad) == UNSUPPORTED, bad
    for bad in (dict(c=CACHE + 8), dict(s=SLOTS + 4), dict(t=TABLE + 2), dict(n=LENS + 1), dict(r=REFS + 2), dict(ws=WS + 8)):
        assert reserve(**bad) == ALIGNMENT, bad
    assert reserve(ws=None) == WORKSPACE and reserve(less=1) == WORKSPACE

    def free(t=TABLE, B=3, W=5, r=REFS, pages=9, rows=OTHER, n=4):
        return dl.brq_kv_free(t, B, W, r, pages, rows, n, None)
    assert free() == 0 and free(rows=None, n=3) == 0 and free(n=0, t=None) == 0 and free(W=0, t=None) == 0
    for bad in (dict(B=-1), dict(W=-1), dict(n=-1), dict(pages=-1), dict(t=None), dict(r=None), dict(rows=None)):
        assert free(**bad) == INVALID, bad
    assert free(B=1 << 20, W=1 << 11) == UNSUPPORTED and free(n=1 << 31) == UNSUPPORTED and free(pages=1 << 31) == UNSUPPORTED
    for k in ("t", "r", "rows"):
        assert free(**{k: TABLE + 2}) == ALIGNMENT, k


i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
i64 = lambda *s: torch.zeros(s, dtype=torch.int64)  # noqa: E731
f32 = lambda *s: torch.zeros(s)  # noqa: E731
PAGE = lambda: u8(3, 2, 16 * 68)  # noqa: E731
CALLS = {
    "brq_tree_attention": (
        lambda a: brq.tree_attention(None, a["q"], a["cache"], a["table"], a["lens"], a["mask"], 16, out=a["out"], lse=a["lse"],
                                     ws=a["ws"]),
        dict(q=f32(3, 5, 4, 64), cache=PAGE(), table=i32(3, 2), lens=i32(3), mask=i64(3, 5), out=f32(3, 5, 4, 64),
             lse=f32(3, 5, 4), ws=u8(64))),
    "brq_kv_move": (lambda a: brq.kv_move(a["cache"], a["src"], a["dst"], 64, 16, ws=a["ws"]),
                    dict(cache=PAGE(), src=i64(7), dst=i64(7), ws=u8(64))),
    "brq_kv_fork": (lambda a: brq.kv_fork(a["table"], a["lens"], a["parents"], a["refs"], a["out"], a["more"]),
                    dict(table=i32(3, 2), lens=i32(3), parents=i32(5), refs=i32(9), out=i32(5, 2), more=i32(5))),
    "brq_kv_reserve": (lambda a: brq.kv_reserve(a["cache"], a["table"], a["lens"], a["refs"], 6, 64, 16, slots=a["slots"],
                                                ws=a["ws"]),
                       dict(cache=PAGE(), table=i32(4, 2), lens=i32(4), refs=i32(3), slots=i64(4, 6), ws=u8(64))),
    "brq_kv_free": (lambda a: brq.kv_free(a["table"], a["refs"], a["rows"]), dict(table=i32(4, 2), refs=i32(3), rows=i32(2))),
}


class Flat(At):
    """One whose views say the same."""

    def flatten(self, *a):
        return Flat(self._t.flatten(*a), self._gpu)

    def __getitem__(self, i):
        return Flat(self._t[i], self._gpu)


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, a) in CALLS.items() for n in a])
def test_one_tensor_elsewhere(library, call, name):  # noqa: F811
    f, tensors = CALLS[call]
    f({n: Flat(t, 0) for n, t in tensors.items()})
    assert library.called == [call]
    library.called.clear()
    for gpu in (1, -1):
        with pytest.raises(ValueError):
            f({n: Flat(t, gpu if n == name else 0) for n, t in tensors.items()})
    assert not library.called


@pytest.mark.parametrize("call,name,other", [
    ("brq_tree_attention", "q", f32(15, 4, 64)), ("brq_tree_attention", "q", f32(3, 7, 4, 64)[:, :5]),
    ("brq_tree_attention", "q", f32(3, 5, 4, 64).double()), ("brq_tree_attention", "out", f32(3, 5, 4, 128)[..., :64]),
    ("brq_tree_attention", "out", f32(3, 5, 4, 64).half()), ("brq_tree_attention", "mask", i64(3, 4)),
    ("brq_tree_attention", "mask", i32(3, 5)), ("brq_tree_attention", "lens", i64(3)), ("brq_tree_attention", "table", i32(2, 2)),
    ("brq_tree_attention", "lse", f32(15, 4)), ("brq_tree_attention", "ws", u8(64, 2)[:, 0]),
    ("brq_kv_move", "src", i32(7)), ("brq_kv_move", "dst", i64(6)), ("brq_kv_move", "cache", u8(3, 2, 16 * 34)),
    ("brq_kv_fork", "parents", i64(5)), ("brq_kv_fork", "lens", i32(2)), ("brq_kv_fork", "out", i32(5, 3)),
    ("brq_kv_fork", "more", i32(4)), ("brq_kv_fork", "table", i32(6)), ("brq_kv_reserve", "refs", i32(4)),
    ("brq_kv_reserve", "slots", i64(4, 5)), ("brq_kv_reserve", "table", i32(2, 4).t()), ("brq_kv_reserve", "lens", i32(3)),
    ("brq_kv_free", "rows", i64(2)), ("brq_kv_free", "refs", f32(3)), ("brq_kv_free", "table", i32(8))])
def test_other_layouts(library, call, name, other):  # noqa: F811
    f, tensors = CALLS[call]
    with pytest.raises(ValueError):
        f({n: Flat(other if n == name else t, 0) for n, t in tensors.items()})
    assert not library.called

"""CPU checks of the microscaled 4-bit operators: the dry run of their launches
(every index walked against its buffer) and every refusal, with fake device
addresses that are never dereferenced."""

import numpy as np
import pytest

import butterfly_rotation_quantization_amd as brq
import synthetic as S
from test_host_dryrun import DPlan, _ok, dl  # noqa: F401  (dl: the dry-run library)

X, Y, WS, CODES, SCALES = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000
B2, S2, SLOTS, CACHE, TABLE, LENS = (0x60000000 + i * 0x1000000 for i in range(6))
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


def rht(dl, d):
    return DPlan(dl, S.random_plan(np.random.default_rng(d), (2,) * (d.bit_length() - 1), "hadamard"))


@pytest.mark.parametrize("rows,n,d", [(1, 32, 0), (3, 4000, 32), (7, 11008, 128), (5, 768, 256), (64, 4096, 64)])
def test_quantize_walk(dl, rows, n, d):
    p = rht(dl, d) if d else None
    h = p.h if p else None
    for t, ld in ((0, n), (1, n + 8), (2, n)):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_mx_quantize(h, X, t, ld, rows, n, CODES, SCALES, None), f"quantize {rows}x{n}")
        _ok(dl, dl.brq_mx_dequantize(h, CODES, SCALES, rows, n, Y, t, ld, None), f"dequantize {rows}x{n}")
        assert dl.brq_dryrun_launches() == 2


def test_quantize_refusals(dl):
    q = lambda h=None, x=X, t=1, ld=4096, r=4, n=4096, c=CODES, s=SCALES: dl.brq_mx_quantize(h, x, t, ld, r, n, c, s, None)  # noqa: E731
    u = lambda h=None, x=X, t=1, ld=4096, r=4, n=4096, c=CODES, s=SCALES: dl.brq_mx_dequantize(h, c, s, r, n, x, t, ld, None)  # noqa: E731
    for f in (q, u):
        assert f() == 0 and f(r=0) == 0 and f(n=0, x=None) == 0
        assert f(t=3) == INVALID and f(t=-1) == INVALID
        assert f(n=4080) == INVALID and f(ld=4095) == INVALID and f(r=-1) == INVALID and f(n=-32) == INVALID
        assert f(x=None) == INVALID and f(c=None) == INVALID and f(s=None) == INVALID
        assert f(x=X + 8) == ALIGNMENT and f(ld=4100) == ALIGNMENT
        assert f(c=CODES + 8) == ALIGNMENT and f(s=SCALES + 2) == ALIGNMENT
        assert f(r=1 << 40) == UNSUPPORTED
        p16, p512, p64 = rht(dl, 16), rht(dl, 512), rht(dl, 64)
        assert f(h=p16.h) == UNSUPPORTED and f(h=p512.h) == UNSUPPORTED
        assert f(h=p64.h, n=4000) == INVALID  # 64 does not divide 4000
        dense = DPlan(dl, S.random_plan(np.random.default_rng(1), (8, 16), "per_group"))
        assert f(h=dense.h) == UNSUPPORTED
        assert dl.brq_last_error()


MM = [(1, 8192, 28672), (16, 11008, 4000), (17, 130, 96), (333, 4096, 11008), (1, 1, 32), (5, 3, 0), (2049, 513, 160),
      (4096, 8192, 28672), (300, 16384, 256), (64, 128, 65536), (2101, 4197, 768), (50, 8193, 544), (100, 70, 160),
      (1 << 16, 1 << 17, 4096), (70, 1 << 26, 256), (1, 1 << 28, 64), (1 << 17, 1 << 16, 128), (1 << 28, 32, 32), (100, 300, 1 << 23), (65, 128, (1 << 23) + 32)]


@pytest.mark.parametrize("T,m,n", MM)
def test_matmul_walk(dl, T, m, n):
    nb = dl.brq_mx_matmul_workspace_bytes(T, m, n)
    for yt, ldy in ((0, m), (1, m + 3), (2, m)):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_mx_matmul(CODES, SCALES, B2, S2, T, m, n, Y, yt, ldy, WS if nb else None, nb, None),
            f"matmul {T}x{m}x{n}")
        assert dl.brq_dryrun_launches() >= 1
    if nb:
        assert dl.brq_mx_matmul(CODES, SCALES, B2, S2, T, m, n, Y, 1, m, WS, nb - 1, None) == WORKSPACE
        assert dl.brq_mx_matmul(CODES, SCALES, B2, S2, T, m, n, Y, 1, m, None, nb, None) == WORKSPACE
        assert dl.brq_mx_matmul(CODES, SCALES, B2, S2, T, m, n, Y, 1, m, WS + 8, nb, None) == ALIGNMENT


def test_matmul_refusals(dl):
    def f(a=CODES, sa=SCALES, b=B2, sb=S2, T=40, m=96, n=128, y=Y, yt=1, ldy=96):
        nb = dl.brq_mx_matmul_workspace_bytes(T, m, n)
        return dl.brq_mx_matmul(a, sa, b, sb, T, m, n, y, yt, ldy, WS, nb, None)
    assert f() == 0 and f(T=0) == 0 and f(m=0) == 0
    assert f(yt=5) == INVALID and f(n=100) == INVALID and f(ldy=95) == INVALID
    assert f(T=-1) == INVALID and f(m=-1) == INVALID and f(n=-32) == INVALID
    for k in ("a", "sa", "b", "sb", "y"):
        assert f(**{k: None}) == INVALID
    assert f(a=CODES + 4) == ALIGNMENT and f(b=B2 + 8) == ALIGNMENT
    assert f(sa=SCALES + 1) == ALIGNMENT and f(sb=S2 + 2) == ALIGNMENT and f(y=Y + 1) == ALIGNMENT
    assert f(m=1 << 31, ldy=1 << 31) == UNSUPPORTED
    # more threads than a launch can have
    assert f(T=(1 << 28) + 1) == UNSUPPORTED and f(m=(1 << 28) + 1, ldy=1 << 29) == UNSUPPORTED
    assert f(T=1 << 17, m=(1 << 16) + 1, ldy=1 << 17) == UNSUPPORTED and f(n=(1 << 28) + 32) == UNSUPPORTED
    assert dl.brq_mx_matmul_workspace_bytes(1 << 17, (1 << 16) + 1, 128) == 0


def test_page_bytes(dl):
    for D in (64, 128, 256):
        for P in (16, 64, 1024):
            assert dl.brq_kv_page_bytes(D, P) == 2 * P * (D // 2 + D // 32)
    for D, P in ((96, 64), (32, 64), (512, 64), (128, 8), (128, 48), (128, 2048), (128, 0), (128, -16)):
        assert dl.brq_kv_page_bytes(D, P) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 64, 1024])
def test_cache_walk(dl, D, P):
    plan = rht(dl, D)
    for h in (None, plan.h):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_kv_append(h, X, 3 * D, Y, 5 * D, 1, SLOTS, 7, 3, D, P, 11, CACHE, None), "append")
        _ok(dl, dl.brq_kv_read(h, CACHE, SLOTS, 7, 3, D, P, 11, X, 3 * D, Y, 5 * D, 2, None), "read")
        assert dl.brq_dryrun_launches() == 2


def test_cache_refusals(dl):
    def app(h=None, k=X, ldk=1024, v=Y, ldv=1024, t=1, s=SLOTS, n=5, H=8, D=128, P=64, pages=9, c=CACHE):
        return dl.brq_kv_append(h, k, ldk, v, ldv, t, s, n, H, D, P, pages, c, None)

    def read(h=None, k=X, ldk=1024, v=Y, ldv=1024, t=1, s=SLOTS, n=5, H=8, D=128, P=64, pages=9, c=CACHE):
        return dl.brq_kv_read(h, c, s, n, H, D, P, pages, k, ldk, v, ldv, t, None)
    for f in (app, read):
        assert f() == 0 and f(n=0) == 0 and f(pages=0, c=None) == 0
        assert f(t=7) == INVALID and f(n=-1) == INVALID and f(H=0) == INVALID and f(pages=-1) == INVALID
        assert f(ldk=1016) == INVALID and f(ldv=1016) == INVALID
        for k in "kvsc":
            assert f(**{k: None}) == INVALID
        assert f(D=96, H=1) == UNSUPPORTED and f(P=24) == UNSUPPORTED and f(n=1 << 31) == UNSUPPORTED
        assert f(k=X + 8) == ALIGNMENT and f(ldv=1028) == ALIGNMENT and f(c=CACHE + 4) == ALIGNMENT
        assert f(s=SLOTS + 4) == ALIGNMENT
        p = rht(dl, 64)
        assert f(h=p.h) == UNSUPPORTED  # d must be the head dimension


@pytest.mark.parametrize("B,hq,H,D,P", [(1, 32, 8, 128, 64), (96, 64, 8, 128, 32), (3, 7, 1, 64, 16),
                                        (2, 40, 2, 256, 1024), (4, 4, 4, 256, 128), (1, 128, 1, 128, 64)])
def test_attention_walk(dl, B, hq, H, D, P):
    plan = rht(dl, D)
    nb = dl.brq_paged_attention_workspace_bytes(B, hq, H, D)
    for h, lse in ((None, None), (plan.h, SCALES)):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_paged_attention(h, X, hq * D, 1, CACHE, 100, TABLE, 40, LENS, B, hq, H, D, P, 0.1, 0, Y, hq * D,
                                       lse, WS if nb else None, nb, None), "attention")
        assert dl.brq_dryrun_launches() == 1
    if nb:
        assert dl.brq_paged_attention(None, X, hq * D, 1, CACHE, 100, TABLE, 40, LENS, B, hq, H, D, P, 0.1, 0, Y,
                                      hq * D, None, WS, nb - 1, None) == WORKSPACE


def test_attention_refusals(dl):
    def f(h=None, q=X, ldq=4096, t=1, c=CACHE, pages=9, tb=TABLE, ldt=4, ln=LENS, B=2, hq=32, H=8, D=128, P=64,
          scale=0.1, window=0, o=Y, ldo=4096, lse=None, ws=WS):
        nb = dl.brq_paged_attention_workspace_bytes(B, hq, H, D) if H > 0 else 0
        return dl.brq_paged_attention(h, q, ldq, t, c, pages, tb, ldt, ln, B, hq, H, D, P, scale, window, o, ldo, lse,
                                      ws, nb, None)
    assert f() == 0 and f(B=0) == 0 and f(ldt=0, tb=None) == 0 and f(pages=0, c=None) == 0 and f(window=5) == 0
    assert f(t=9) == INVALID and f(B=-1) == INVALID and f(H=0) == INVALID and f(hq=12) == INVALID
    assert f(hq=0) == INVALID and f(window=-1) == INVALID and f(ldt=-1) == INVALID and f(pages=-1) == INVALID
    assert f(scale=float("nan")) == INVALID and f(scale=float("inf")) == INVALID
    assert f(ldq=4088) == INVALID and f(ldo=4088) == INVALID
    for k in ("q", "c", "tb", "ln", "o"):
        assert f(**{k: None}) == INVALID
    assert f(D=96) == UNSUPPORTED and f(P=40) == UNSUPPORTED and f(B=1 << 24) == UNSUPPORTED
    assert f(q=X + 4) == ALIGNMENT and f(ldo=4098) == ALIGNMENT and f(c=CACHE + 8) == ALIGNMENT
    assert f(tb=TABLE + 2) == ALIGNMENT and f(lse=SCALES + 1) == ALIGNMENT
    p = rht(dl, 64)
    assert f(h=p.h) == UNSUPPORTED
    assert f(ws=None) == WORKSPACE




@pytest.mark.parametrize("B,hq,H", [(4097, 64, 64), (4096, 4095, 4095), ((1 << 24) - 1, 1, 1), (1 << 23, 1, 1), (5000, 3355, 1),
                                    (4096, 4080, 255), (100000, 160, 8)])
def test_attention_walk_of_large_batches(dl, B, hq, H):
    """Up to the largest number of sequences times query heads every launch has
    fewer than 2^32 threads."""
    nb = dl.brq_paged_attention_workspace_bytes(B, hq, H, 256)
    for D in (64, 256):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_paged_attention(None, X, hq * D, 1, CACHE, 100, TABLE, 4, LENS, B, hq, H, D, 16, 0.1, 0, Y, hq * D,
                                       None, WS if nb else None, nb, None), f"attention {B}x{hq}/{H}")


def test_attention_refuses_a_launch_that_cannot_be(dl):
    for B, hq in ((1 << 24, 1), (1 << 20, 16), (4096, 4096), (1 << 23, 2)):
        for D in (64, 128):
            nb = dl.brq_paged_attention_workspace_bytes(B, hq, hq, D)
            assert dl.brq_paged_attention(None, X, hq * D, 1, CACHE, 9, TABLE, 4, LENS, B, hq, hq, D, 64, 0.1, 0, Y, hq * D,
                                          None, WS, nb, None) == UNSUPPORTED

"""CPU checks of the products with an epilogue: the dry run of their launches,
every refusal with fake device addresses that are never dereferenced, and the
binding with tensors that only say where they are."""

import ctypes

import pytest
import torch

import butterfly_rotation_quantization_amd as brq
from test_host_dryrun import _ok, dl  # noqa: F401  (dl: the dry-run library)
from test_host_mx import ALIGNMENT, B2, CODES, INVALID, S2, SCALES, UNSUPPORTED, WORKSPACE, WS, Y
from test_host_mx_binding import At, library, u8  # noqa: F401

BIAS, MUL, RES = 0x1000000000, 0x1100000000, 0x1200000000


def epilogue(**kw):
    full = dict(bias=BIAS, mul=MUL, residual=RES, ldmul=4096, ldresidual=4096, act=4, bias_type=1, mul_type=1,
                residual_type=1)
    return ctypes.byref(brq.MxEpilogue(**{**full, **kw}))


@pytest.mark.parametrize("T,m,n", [(1, 8192, 28672), (50, 8193, 544), (333, 4096, 11008), (4096, 8192, 28672),
                                   (100, 70, 160), (5, 3, 0), (300, 385, 16640)])
def test_linear_walk(dl, T, m, n):  # noqa: F811
    nb = dl.brq_mx_matmul_workspace_bytes(T, m, n)
    for ep in (None, epilogue(ldmul=m, ldresidual=m + 3), epilogue(bias=None, mul=None, ldmul=0, ldresidual=m)):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_mx_linear(CODES, SCALES, B2, S2, T, m, n, ep, Y, 1, m, WS, nb, None), f"linear {T}x{m}x{n}")
        assert dl.brq_dryrun_launches() == 1


def test_linear_refusals(dl):  # noqa: F811
    nb = dl.brq_mx_matmul_workspace_bytes(333, 4096, 11008)
    f = lambda ep=None, T=333, m=4096, n=11008, a=CODES, y=Y, t=1, ld=4096, ws=WS, nb=nb, **kw: \
        dl.brq_mx_linear(a, SCALES, B2, S2, T, m, n, ep or epilogue(**kw), y, t, ld, ws, nb, None)  # noqa: E731
    assert f() == 0 and f(T=0) == 0 and f(m=0) == 0
    for bad in (dict(act=5), dict(act=-1), dict(bias_type=3), dict(mul_type=-1), dict(residual_type=7),
                dict(ldmul=4095), dict(ldresidual=0), dict(t=3), dict(ld=4095), dict(n=11000), dict(T=-1),
                dict(a=None), dict(y=None)):
        assert f(**bad) == INVALID, bad
    # a part that is not there is not looked at
    assert f(bias=None, bias_type=9, mul=None, mul_type=9, ldmul=0, residual=None, residual_type=9, ldresidual=0) == 0
    for bad in (dict(bias=BIAS + 1), dict(mul=MUL + 1), dict(residual=RES + 2, residual_type=0), dict(y=Y + 1)):
        assert f(**bad) == ALIGNMENT, bad
    assert f(bias=BIAS + 2, mul=MUL + 2, residual=RES + 2) == 0
    assert f(T=1 << 29) == UNSUPPORTED
    assert f(ws=None) == WORKSPACE and f(nb=nb - 1) == WORKSPACE and f(ws=WS + 8) == ALIGNMENT
    assert dl.brq_last_error()


f32 = lambda *s: torch.zeros(s)  # noqa: E731
LINEAR = (lambda t: brq.mx_linear(t["a"], t["sa"], t["b"], t["sb"], bias=t["bias"], act="silu", mul=t["mul"],
                                  residual=t["residual"], y=t["y"], ws=t["ws"]),
          dict(a=u8(4, 32), sa=u8(4, 2), b=u8(7, 32), sb=u8(7, 2), bias=f32(7), mul=f32(4, 7), residual=f32(4, 7),
               y=f32(4, 7), ws=u8(64)))


@pytest.mark.parametrize("name", list(LINEAR[1]))
def test_linear_one_tensor_elsewhere(library, name):  # noqa: F811
    f, tensors = LINEAR
    f({n: At(t, 0) for n, t in tensors.items()})
    assert library.called == ["brq_mx_linear"]
    library.called.clear()
    for gpu in (1, -1):
        with pytest.raises(ValueError):
            f({n: At(t, gpu if n == name else 0) for n, t in tensors.items()})
    assert not library.called


@pytest.mark.parametrize("name,other", [("a", u8(4, 30)), ("sb", u8(6, 2)), ("bias", f32(6)), ("bias", f32(7).double()),
                                        ("bias", f32(14)[::2]), ("mul", f32(4, 6)), ("mul", f32(7, 4).t()),
                                        ("residual", f32(7)), ("residual", f32(4, 7).int()), ("y", f32(4, 8)),
                                        ("y", f32(4, 7).double()), ("ws", u8(64, 2)[:, 0])])
def test_linear_other_layouts(library, name, other):  # noqa: F811
    f, tensors = LINEAR
    with pytest.raises(ValueError):
        f({n: At(other if n == name else t, 0) for n, t in tensors.items()})
    assert not library.called


def test_linear_passes_what_it_is_given(library, monkeypatch):  # noqa: F811
    seen = []
    monkeypatch.setattr(library, "brq_mx_linear", lambda *a: seen.append(a[7]) or 0, raising=False)
    f, t = LINEAR[0], {n: At(x, 0) for n, x in LINEAR[1].items()}
    t["mul"] = At(torch.zeros((4, 12), dtype=torch.bfloat16)[:, :7], 0)
    f(t)
    e = seen[0]._obj
    assert (e.bias, e.mul, e.residual) == tuple(t[n].data_ptr() for n in ("bias", "mul", "residual"))
    assert (e.act, e.bias_type, e.mul_type, e.residual_type, e.ldmul, e.ldresidual) == (4, 0, 1, 0, 12, 7)
    brq.mx_linear(t["a"], t["sa"], t["b"], t["sb"], y=t["y"], ws=t["ws"])
    assert seen[1] is None
    with pytest.raises(ValueError, match="act"):
        brq.mx_linear(t["a"], t["sa"], t["b"], t["sb"], act="tanh", y=t["y"], ws=t["ws"])


OFFS = 0x1300000000
# one group and many, more groups than rows, rows too short and too long for tiles, streams and tiles of either size
GROUPED = [(1, 1, 1, 32), (5, 300, 70, 160), (777, 64, 1376, 2048), (32, 8, 11008, 4096), (8192, 8, 4096, 11008),
           (3000, 8, 513, 544), (1 << 20, 16, 300, 768), (1 << 16, 1, 1 << 16, 256), (1000, 1 << 20, 64, 64), (90, 2, 64, 0),
           (70, 1, 64, (1 << 23) + 32), (4096, 64, 16384, 288), (2000, 2, 100, 1 << 23)]


@pytest.mark.parametrize("T,E,m,n", GROUPED)
def test_grouped_walk(dl, T, E, m, n):  # noqa: F811
    nb = dl.brq_mx_grouped_matmul_workspace_bytes(T, E, m, n)
    ws = WS if nb else None
    for ep in (None, epilogue(ldmul=m, ldresidual=m + 3)):
        dl.brq_dryrun_reset()
        _ok(dl, dl.brq_mx_grouped_matmul(CODES, SCALES, B2, S2, OFFS, T, E, m, n, ep, Y, 1, m, ws, nb, None),
            f"grouped {T}x{E}x{m}x{n}")
        assert dl.brq_dryrun_launches() == 1
    if nb:
        g = lambda ws, nb: dl.brq_mx_grouped_matmul(CODES, SCALES, B2, S2, OFFS, T, E, m, n, None, Y, 1, m, ws, nb, None)  # noqa: E731
        assert g(WS, nb - 1) == WORKSPACE and g(None, nb) == WORKSPACE and g(WS + 8, nb) == ALIGNMENT


def test_grouped_refusals(dl):  # noqa: F811
    def f(a=CODES, sa=SCALES, b=B2, sb=S2, offs=OFFS, T=40, E=3, m=96, n=128, ep=None, y=Y, t=1, ld=96):
        nb = dl.brq_mx_grouped_matmul_workspace_bytes(T, E, m, n)
        return dl.brq_mx_grouped_matmul(a, sa, b, sb, offs, T, E, m, n, ep, y, t, ld, WS, nb, None)
    assert f() == 0 and f(T=0) == 0 and f(m=0) == 0 and f(E=0, b=None, sb=None, offs=None) == 0
    assert f(t=5) == INVALID and f(n=100) == INVALID and f(ld=95) == INVALID and f(E=-1) == INVALID
    assert f(T=-1) == INVALID and f(m=-1) == INVALID and f(n=-32) == INVALID
    for k in ("a", "sa", "b", "sb", "y", "offs"):
        assert f(**{k: None}) == INVALID, k
    assert f(a=CODES + 4) == ALIGNMENT and f(sb=S2 + 2) == ALIGNMENT and f(y=Y + 1) == ALIGNMENT and f(offs=OFFS + 2) == ALIGNMENT
    assert f(ep=epilogue(ldmul=95)) == INVALID and f(ep=epilogue(act=9)) == INVALID and f(ep=epilogue(bias=BIAS + 1)) == ALIGNMENT
    assert f(E=(1 << 20) + 1) == UNSUPPORTED and f(T=(1 << 28) + 1) == UNSUPPORTED
    assert f(T=1 << 20, E=1 << 20, m=1 << 10, ld=1 << 10) == UNSUPPORTED  # more threads than a launch can have
    assert dl.brq_mx_grouped_matmul_workspace_bytes(1 << 20, 1 << 20, 1 << 10, 512) == 0


GROUP = (lambda t: brq.mx_grouped_matmul(t["a"], t["sa"], t["b"], t["sb"], t["offs"], bias=t["bias"], act="gelu",
                                         mul=t["mul"], residual=t["residual"], y=t["y"], ws=t["ws"]),
         dict(a=u8(4, 32), sa=u8(4, 2), b=u8(3, 7, 32), sb=u8(3, 7, 2), offs=torch.zeros(4, dtype=torch.int32),
              bias=f32(3, 7), mul=f32(4, 7), residual=f32(4, 7), y=f32(4, 7), ws=u8(64)))


@pytest.mark.parametrize("name", list(GROUP[1]))
def test_grouped_one_tensor_elsewhere(library, name):  # noqa: F811
    f, tensors = GROUP
    f({n: At(t, 0) for n, t in tensors.items()})
    assert library.called == ["brq_mx_grouped_matmul"]
    library.called.clear()
    for gpu in (1, -1):
        with pytest.raises(ValueError):
            f({n: At(t, gpu if n == name else 0) for n, t in tensors.items()})
    assert not library.called


@pytest.mark.parametrize("name,other", [("a", u8(4, 30)), ("b", u8(7, 32)), ("sb", u8(3, 6, 2)), ("bias", f32(7)),
                                        ("offs", torch.zeros(3, dtype=torch.int32)), ("offs", torch.zeros(4)),
                                        ("mul", f32(4, 6)), ("residual", f32(7)), ("y", f32(4, 8)), ("ws", u8(64, 2)[:, 0])])
def test_grouped_other_layouts(library, name, other):  # noqa: F811
    f, tensors = GROUP
    with pytest.raises(ValueError):
        f({n: At(other if n == name else t, 0) for n, t in tensors.items()})
    assert not library.called

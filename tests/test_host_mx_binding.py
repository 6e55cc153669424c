"""CPU checks of the microscaled operators' binding: every tensor of a call has
to be on one GPU, a workspace too.  The tensors are stand-ins that say where
they are, and the library is one that only notes that it was called."""

import pytest
import torch

import butterfly_rotation_quantization_amd as brq


class At:
    """A tensor said to be on GPU `gpu` (-1: in host memory)."""

    def __init__(self, t, gpu):
        self._t, self._gpu = t, gpu

    def get_device(self):
        return self._gpu

    @property
    def is_cuda(self):
        return self._gpu >= 0

    @property
    def device(self):
        return f"cuda:{self._gpu}" if self._gpu >= 0 else "cpu"

    def __getattr__(self, name):
        return getattr(self._t, name)


class Library:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(brq, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return lib


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


KV = lambda: torch.zeros((5, 2, 64))  # noqa: E731
CACHE = lambda: u8(3, 2, 16 * 68)  # noqa: E731
CALLS = {
    "quantize": (lambda a: brq.mx_quantize(None, a["x"], a["codes"], a["scales"]),
                 dict(x=torch.zeros((4, 64)), codes=u8(4, 32), scales=u8(4, 2))),
    "dequantize": (lambda a: brq.mx_dequantize(None, a["codes"], a["scales"], out=a["out"]),
                   dict(out=torch.zeros((4, 64)), codes=u8(4, 32), scales=u8(4, 2))),
    "matmul": (lambda a: brq.mx_matmul(a["a"], a["sa"], a["b"], a["sb"], y=a["y"], ws=a["ws"]),
               dict(a=u8(4, 32), sa=u8(4, 2), b=u8(7, 32), sb=u8(7, 2), y=torch.zeros((4, 7)), ws=u8(64))),
    "append": (lambda a: brq.kv_append(None, a["k"], a["v"], a["slots"], a["cache"], 16),
               dict(k=KV(), v=KV(), slots=torch.arange(5), cache=CACHE())),
    "read": (lambda a: brq.kv_read(None, a["cache"], a["slots"], 64, 16, k=a["k"], v=a["v"]),
             dict(k=KV(), v=KV(), slots=torch.arange(5), cache=CACHE())),
    "attention": (lambda a: brq.paged_attention(None, a["q"], a["cache"], a["table"], a["lens"], 16, out=a["out"],
                                                lse=a["lse"], ws=a["ws"]),
                  dict(q=torch.zeros((3, 4, 64)), cache=CACHE(), table=torch.zeros((3, 2), dtype=torch.int32),
                       lens=torch.zeros(3, dtype=torch.int32), out=torch.zeros((3, 4, 64)), lse=torch.zeros((3, 4)),
                       ws=u8(64))),
}


@pytest.mark.parametrize("call,name,gpu", [(c, n, g) for c, (_, a) in CALLS.items() for n in a for g in (1, -1)])
def test_one_tensor_elsewhere(library, call, name, gpu):
    f, tensors = CALLS[call]
    f({n: At(t, 0) for n, t in tensors.items()})
    assert library.called
    library.called.clear()
    with pytest.raises(ValueError):
        f({n: At(t, gpu if n == name else 0) for n, t in tensors.items()})
    assert not library.called


@pytest.mark.parametrize("call", list(CALLS))
def test_all_tensors_on_another_gpu_than_the_current_one(library, call):
    f, tensors = CALLS[call]
    with pytest.raises(ValueError):
        f({n: At(t, 1) for n, t in tensors.items()})
    assert not library.called


@pytest.mark.parametrize("call", ["matmul", "attention"])
def test_a_workspace_with_gaps(library, call):
    """Its elements would count for more bytes in a row than it has."""
    f, tensors = CALLS[call]
    with pytest.raises(ValueError):
        f({n: At(u8(64, 2)[:, 0] if n == "ws" else t, 0) for n, t in tensors.items()})
    assert not library.called


def test_the_stride_of_a_single_row_does_not_matter(library, monkeypatch):
    """A row of a tensor whose rows are no multiple of 16 bytes apart: the
    library is told the row's own length, which it takes."""
    seen = {}
    for name in ("brq_mx_quantize", "brq_mx_dequantize", "brq_mx_matmul", "brq_kv_append", "brq_paged_attention"):
        monkeypatch.setattr(library, name, lambda *a, name=name: seen.update({name: a}) or 0, raising=False)
    wide = torch.zeros((3, 68))[1:2, :64]
    heads = torch.zeros((3, 132))[1:2, :128].unflatten(1, (2, 64))
    g = lambda t: At(t, 0)  # noqa: E731
    codes, scales = g(u8(1, 32)), g(u8(1, 2))
    brq.mx_quantize(None, g(wide), codes, scales)
    brq.mx_dequantize(None, codes, scales, out=g(wide))
    brq.mx_matmul(codes, scales, g(u8(64, 32)), g(u8(64, 2)), y=g(wide), ws=g(u8(64)))
    brq.kv_append(None, g(heads), g(heads), g(torch.zeros(1, dtype=torch.int64)), g(CACHE()), 16)
    brq.paged_attention(None, g(heads), g(CACHE()), g(torch.zeros((1, 2), dtype=torch.int32)),
                        g(torch.zeros(1, dtype=torch.int32)), 16, out=g(heads), ws=g(u8(64)))
    assert seen["brq_mx_quantize"][3] == 64 and seen["brq_mx_dequantize"][7] == 64 and seen["brq_mx_matmul"][9] == 64
    assert seen["brq_kv_append"][2] == 128 and seen["brq_kv_append"][4] == 128
    assert seen["brq_paged_attention"][2] == 128 and seen["brq_paged_attention"][17] == 128


def test_a_window_beyond_32_bits(library, monkeypatch):
    """The C call takes 32 bits: a longer window sees all there is, as its value
    says, and a negative one stays negative (and is refused)."""
    import ctypes
    seen = []
    monkeypatch.setattr(library, "brq_paged_attention", lambda *a: seen.append(ctypes.c_int32(a[15]).value) or 0,
                        raising=False)
    f, tensors = CALLS["attention"]
    t = {n: At(x, 0) for n, x in tensors.items()}
    for window in (0, 5, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, -1, -2 ** 32):
        brq.paged_attention(None, t["q"], t["cache"], t["table"], t["lens"], 16, window=window, out=t["out"], ws=t["ws"])
    assert seen == [0, 5] + [2 ** 31 - 1] * 4 + [-1] * 2


@pytest.mark.parametrize("call,name", [("quantize", "x"), ("dequantize", "out"), ("matmul", "y"), ("append", "kv"),
                                       ("read", "kv"), ("attention", "q out")])
def test_other_types_are_refused_like_other_layouts(library, call, name):
    f, tensors = CALLS[call]
    names = ["k", "v"] if name == "kv" else name.split()
    with pytest.raises(ValueError):
        f({n: At(t.double() if n in names else t, 0) for n, t in tensors.items()})
    assert not library.called

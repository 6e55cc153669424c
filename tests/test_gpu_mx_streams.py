"""The microscaled operators called with a stream other than the current one:
what the binding makes for a call comes from that stream's memory, so it is
neither still in use by the current stream's work nor handed out there while the
call is ahead.  The other stream is kept busy by a sleeping kernel, so that
everything the host does meanwhile comes before the calls' kernels."""

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # cycles: some 0.1 s


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def apart(xs, ys):
    return all(b <= c or d <= a for a, b in spans(xs) for c, d in spans(ys))


def inputs():
    import butterfly_rotation_quantization_amd as brq
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((300, 4096), generator=g, device="cuda").to(torch.bfloat16)
    w = brq.mx_quantize(None, torch.randn((512, 4096), generator=g, device="cuda"))
    cache = brq.kv_cache(8, 2, 128, 64)
    kv = torch.randn((400, 2, 128), generator=g, device="cuda")
    slots = torch.arange(400, device="cuda")
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    lens = torch.tensor([70, 128, 1], dtype=torch.int32, device="cuda")
    q = torch.randn((3, 8, 128), generator=g, device="cuda")
    return x, w, cache, kv, slots, table, lens, q


def calls(stream):
    """Every call with nothing but its inputs given, temporaries and all."""
    import butterfly_rotation_quantization_amd as brq
    x, w, cache, kv, slots, table, lens, q = inputs()
    import torch
    torch.cuda.synchronize()

    def run():
        y = brq.mx_matmul(*brq.mx_quantize(None, x, stream=stream), *w, stream=stream)
        back = brq.mx_dequantize(None, *brq.mx_quantize(None, x, stream=stream), stream=stream)
        brq.kv_append(None, kv, kv, slots, cache, 64, stream=stream)
        k, v = brq.kv_read(None, cache, slots, 128, 64, stream=stream)
        out = brq.paged_attention(None, q, cache, table, lens, 64, stream=stream)
        return y, back, k, v, out
    return run


@pytest.mark.parametrize("raw", [False, True])
def test_temporaries_outlive_the_calls(raw):
    import torch
    announce(f"mx calls on a busy stream raw={raw}")
    want = calls(None)()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    run = calls(s.cuda_stream if raw else s)
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = run()
    # the current stream overwrites all the memory that it is given
    junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
            for n in (300 * 2048, 300 * 128, 300 * 4096 * 2, 300 * 512 * 2, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
    assert not s.query(), "the stream was to be busy still"
    assert apart(junk, got)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_memory_the_current_stream_still_uses_is_not_taken():
    """Tensors freed with the current stream's work on them ahead: the calls on
    another stream, which does not wait for that work, get other memory."""
    import torch
    announce("mx calls beside a busy current stream")
    s = torch.cuda.Stream()
    run = calls(s)
    run()
    torch.cuda.synchronize()
    sizes = [(300, 2048), (300, 128), (300, 512), (300, 4096), (400, 2, 128), (3, 8, 128)]
    freed = [torch.zeros(z, dtype=t, device="cuda") for z in sizes for t in (torch.uint8, torch.bfloat16, torch.float32)]
    torch.cuda._sleep(BUSY)
    for t in freed:
        t.add_(1)
    where = spans(freed)
    del freed, t
    got = run()
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy still"
    assert all(b <= c or d <= a for a, b in spans(got) for c, d in where)
    torch.cuda.synchronize()


def test_the_default_stream_by_number():
    """Stream 0 is the default stream, which torch's current one is here."""
    import torch
    announce("mx calls on stream 0")
    want = calls(None)()
    got = calls(0)()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)

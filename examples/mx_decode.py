"""One attention layer served in the microscaled 4-bit format: weights,
activations and key-value cache all in blocks of 32 four-bit values with a
shared scale, rotated so that no value of a block stands out.

    python examples/mx_decode.py [--hidden 4096] [--q-heads 32] [--heads 8]
        [--head-dim 128] [--batch 16] [--tokens 2048] [--steps 16]

A prompt's keys and values are projected (mx_quantize, mx_matmul) and appended
to a paged cache (kv_append); a decoding step projects one token a sequence,
appends it, attends over the cache (paged_attention) and projects back.  A step
launches on the current stream and reads its lengths on the device, so it is
captured once and replayed while the sequences grow; the operators allocate
nothing in it, since it gives them their outputs and workspaces.  The
result is compared with the layer computed densely in float32, and each stage
with the same stage in float32 on the stage's own 4-bit operands."""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import butterfly_rotation_quantization_amd as brq  # noqa: E402


def hadamard(d, seed):
    """The rotation H D / sqrt(d) with random signs D."""
    signs = (np.random.default_rng(seed).integers(0, 2, d) * 2 - 1).astype(np.int8)
    return brq.Plan(d, (2,) * (d.bit_length() - 1), "hadamard", signs=signs)


class Weight:
    """A weight [m, n] and what a product of up to T rows with it needs."""

    def __init__(self, w, plan, T):
        self.plan, (self.m, self.n) = plan, w.shape
        self.codes, self.scales = brq.mx_quantize(plan, w)
        # shorter products may need more than longer ones, since they split n
        self.ws = {t: brq.mx_matmul_workspace(t, self.m, self.n) for t in T}

    def __call__(self, x, buffers=None, y=None):
        """x [T, n] times the weight's transpose; buffers: codes and scales of x."""
        codes, scales = brq.mx_quantize(self.plan, x, *(buffers or (None, None)))
        return brq.mx_matmul(codes, scales, self.codes, self.scales, y=y, ws=self.ws.get(x.shape[0]))

    def values(self):
        return brq.mx_dequantize(self.plan, self.codes, self.scales)


class Layer:
    def __init__(self, wqkv, wo, q_heads, heads, head_dim, batch, tokens, page=64):
        self.hq, self.h, self.D, self.page, self.B = q_heads, heads, head_dim, page, batch
        rot = hadamard(128, 0)
        self.qkv, self.o = Weight(wqkv, rot, (batch,)), Weight(wo, rot, (batch,))
        self.rot = hadamard(head_dim, 1)
        per = (tokens + page - 1) // page  # pages of a sequence
        self.cache = brq.kv_cache(batch * per, heads, head_dim, page)
        order = np.random.default_rng(2).permutation(batch * per).reshape(batch, per)
        self.table = torch.from_numpy(order.astype(np.int32)).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        # what a step writes
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        mx = lambda n: (new(batch, n // 2, dtype=torch.uint8), new(batch, n // 32, dtype=torch.uint8))  # noqa: E731
        self.x, self.y, self.x4, self.a4 = new(batch, wqkv.shape[1]), new(batch, wo.shape[0]), mx(wqkv.shape[1]), mx(wo.shape[1])
        self.p, self.a = new(batch, wqkv.shape[0]), new(batch, q_heads, head_dim)
        self.ws = brq.paged_attention_workspace(batch, q_heads, heads, head_dim)

    def heads_of(self, p):
        """Queries, keys and values [tokens, heads, D] of projected rows (views)."""
        q, k, v = p.split((self.hq * self.D, self.h * self.D, self.h * self.D), dim=1)
        return q.unflatten(1, (self.hq, self.D)), k.unflatten(1, (self.h, self.D)), v.unflatten(1, (self.h, self.D))

    def slots(self, seq, at):
        """Cache slots of tokens `at` of sequences `seq`."""
        return self.table[seq, at // self.page].long() * self.page + at % self.page

    def prompt(self, b, x):
        """The first tokens of sequence b: x [tokens, hidden]."""
        _, k, v = self.heads_of(self.qkv(x))
        at = torch.arange(x.shape[0], device="cuda")
        brq.kv_append(self.rot, k, v, self.slots(torch.full_like(at, b), at), self.cache, self.page)
        self.lens[b] = x.shape[0]

    def step(self):
        """One token a sequence: self.x [batch, hidden] to self.y."""
        q, k, v = self.heads_of(self.qkv(self.x, self.x4, self.p))
        seq = torch.arange(self.B, device="cuda")
        brq.kv_append(self.rot, k, v, self.slots(seq, self.lens.long()), self.cache, self.page)
        self.lens.add_(1)
        brq.paged_attention(self.rot, q, self.cache, self.table, self.lens, self.page, out=self.a, ws=self.ws)
        self.o(self.a.flatten(1), self.a4, self.y)


def attend(q, k, v):
    """float32 attention of q [hq, D] over k, v [tokens, h, D]."""
    g = q.shape[0] // k.shape[1]
    k, v = k.repeat_interleave(g, 1).transpose(0, 1), v.repeat_interleave(g, 1).transpose(0, 1).contiguous()
    p = torch.softmax((k * q[:, None]).sum(-1) * q.shape[-1] ** -0.5, dim=-1)
    return (p[..., None] * v).sum(1)


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def stage_errors(layer):
    """Relative error of each stage of the last step against float32 on its own
    4-bit operands."""
    x = brq.mx_dequantize(layer.qkv.plan, *layer.x4)
    a = brq.mx_dequantize(layer.o.plan, *layer.a4)
    q = layer.heads_of(layer.p)[0].float()
    rows = []
    for b in range(layer.B):
        at = torch.arange(int(layer.lens[b]), device="cuda")
        k, v = brq.kv_read(layer.rot, layer.cache, layer.slots(torch.full_like(at, b), at), layer.D, layer.page,
                           out_dtype=torch.float32)
        rows.append(attend(q[b], k, v))
    return {"projection": off(layer.p, x @ layer.qkv.values().t()), "attention": off(layer.a, torch.stack(rows)),
            "output": off(layer.y, a @ layer.o.values().t())}


def run(hidden=4096, q_heads=32, heads=8, head_dim=128, batch=16, tokens=2048, steps=16, timed=50, seed=0):
    """Returns the stages' errors, the error against the dense layer and the
    time of a captured step in microseconds."""
    torch.manual_seed(seed)
    rng = np.random.default_rng(seed)
    rand = lambda *s: (torch.randn(s, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    wqkv, wo = rand((q_heads + 2 * heads) * head_dim, hidden), rand(hidden, q_heads * head_dim)
    layer = Layer(wqkv, wo, q_heads, heads, head_dim, batch, tokens + steps + 1)
    lens = [int(n) for n in rng.integers(max(1, tokens // 8), tokens + 1, batch)]
    seen = [torch.randn(n, hidden, device="cuda").bfloat16() for n in lens]
    for b, x in enumerate(seen):
        layer.prompt(b, x)
    fresh = torch.randn(steps, batch, hidden, device="cuda").bfloat16()

    # one step eagerly, the rest by replaying a captured one
    layer.x.copy_(fresh[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()  # recorded, not run
    for i in range(1, steps):
        layer.x.copy_(fresh[i])
        graph.replay()
    errors = stage_errors(layer)

    # the same layer, dense: float32 throughout
    rows = []
    for b in range(batch):
        xs = torch.cat([seen[b], fresh[:, b]]).float()
        q, k, v = layer.heads_of(xs @ wqkv.float().t())
        rows.append(attend(q[-1], k, v).flatten())
    errors["dense"] = off(layer.y, torch.stack(rows) @ wo.float().t())

    full = layer.lens.clone()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(timed):
        layer.lens.copy_(full - 1)  # the last token again
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    return errors, t0.elapsed_time(t1) * 1e3 / max(1, timed)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("hidden", 4096), ("q-heads", 32), ("heads", 8), ("head-dim", 128), ("batch", 16),
                          ("tokens", 2048), ("steps", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    errors, us = run(a.hidden, a.q_heads, a.heads, a.head_dim, a.batch, a.tokens, a.steps)
    for name, e in errors.items():
        what = "the dense float32 layer" if name == "dense" else "float32 on the same 4-bit operands"
        print(f"{name:<11} {e:.2e} off {what}")
    print(f"a step of {a.batch} sequences of up to {a.tokens + a.steps} tokens: {us:.1f} us")


if __name__ == "__main__":
    main()

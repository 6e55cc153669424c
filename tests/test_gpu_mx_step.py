"""The operators of a drafted step run together, as a server runs them, and on
other streams than the current one, two at a time, and in captured graphs."""

import numpy as np
import pytest

from gpu_util import announce
from oracle import mx as X
from test_gpu_kv import rht
from test_gpu_kv_tree import to_mask
from test_gpu_mx_streams import BUSY

pytestmark = pytest.mark.gpu

# a small model's layer: width, query and key-value heads, their dimension, experts and their width
W, HQ, H, D, E, M, P = 512, 8, 2, 64, 4, 384, 16


class Layer:
    """Attention with its projections, then two of four experts for each token, in the 4-bit format throughout."""

    def __init__(self, seed):
        import butterfly_rotation_quantization_amd as brq
        import torch
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        weight = lambda *s: brq.mx_quantize(None, self.rand(*s) / s[-1] ** 0.5)  # noqa: E731
        self.qkv, self.o = weight((HQ + 2 * H) * D, W), weight(W, HQ * D)
        self.bias = self.rand((HQ + 2 * H) * D) * 0.1
        up, down = weight(E * M, W), weight(E * W, M)
        self.up, self.down = [z.view(E, M, -1) for z in up], [z.view(E, W, -1) for z in down]
        self.plan, _ = rht(D)

    def rand(self, *s):
        import torch
        return torch.randn(s, generator=self.g, device="cuda")

    def heads(self, x):
        """q, k, v of rows x [n, W]."""
        import butterfly_rotation_quantization_amd as brq
        import torch
        y = brq.mx_linear(*brq.mx_quantize(None, x), *self.qkv, bias=self.bias, out_dtype=torch.float32)
        return [z.unflatten(1, (-1, D)) for z in y.split([HQ * D, H * D, H * D], dim=1)]

    def after(self, x, attended, expert):
        """The layer's output: row i takes experts expert[i] and (expert[i] + 1) % E, each half."""
        import butterfly_rotation_quantization_amd as brq
        import torch
        n = x.shape[0]
        y = brq.mx_linear(*brq.mx_quantize(None, attended.reshape(n, HQ * D)), *self.o, residual=x, out_dtype=torch.float32)
        pick = torch.cat((expert, (expert + 1) % E))
        order = torch.sort(pick, stable=True).indices
        counts = (pick[:, None] == torch.arange(E, device="cuda")).sum(0)
        offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
        rows = order % n
        h = brq.mx_grouped_matmul(*brq.mx_quantize(None, y[rows]), *self.up, offsets, act="silu", out_dtype=torch.float32)
        z = brq.mx_grouped_matmul(*brq.mx_quantize(None, h), *self.down, offsets, mul=torch.full((2 * n, W), 0.5, device="cuda"),
                                  out_dtype=torch.float32)
        both = torch.empty_like(z)
        both[order] = z
        return y + both[:n] + both[n:]


def test_a_drafted_step_is_what_single_tokens_give():
    """Two samples of one prompt (pages shared, then copied) verify a tree of six
    drafts each; the accepted path moves to the front.  Each path of the tree, fed
    token by token to a cache of its own, gives the same rows, and the cache
    after the move holds the accepted tokens' bytes."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("a drafted step")
    layer, B, N, n0, pages = Layer(5), 2, 6, 21, 24
    prompt = layer.rand(n0, W)
    cache = brq.kv_cache(pages, H, D, P)
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    _, k, v = layer.heads(prompt)
    brq.kv_append(layer.plan, k.contiguous(), v.contiguous(), brq.kv_reserve(cache, table, lens, refs, n0, D, P).view(-1), cache, P)
    lens += n0
    kids, klens = brq.kv_fork(table, lens, torch.zeros(B, dtype=torch.int32, device="cuda"), refs)
    slots = brq.kv_reserve(cache, kids, klens, refs, N, D, P)
    assert (slots >= 0).all() and len(slots.unique()) == B * N
    parents = [[-1, 0, 0, 1, 2, 4], [-1, -1, 1, 2, 2, 3]]
    masks = []
    for par in parents:
        row = []
        for j, p in enumerate(par):
            row.append((row[p] if p >= 0 else 0) | 1 << j)
        masks.append(row)
    x, expert = layer.rand(B * N, W), torch.arange(B * N, device="cuda") * 7 % E
    q, k, v = layer.heads(x)
    brq.kv_append(layer.plan, k.contiguous(), v.contiguous(), slots.view(-1), cache, P)
    mask = torch.from_numpy(to_mask(masks)).cuda()
    attended = brq.tree_attention(layer.plan, q.reshape(B, N, HQ, D).contiguous(), cache, kids, klens, mask, P)
    out = layer.after(x, attended, expert)

    for b, par in enumerate(parents):
        for leaf in range(N):
            path = [j for j in range(N) if masks[b][leaf] >> j & 1]
            own = brq.kv_cache(3, H, D, P)
            t = torch.arange(3, dtype=torch.int32, device="cuda")[None]
            rows = torch.cat((prompt, x[[b * N + j for j in path]]))
            qs, ks, vs = layer.heads(rows)
            brq.kv_append(layer.plan, ks.contiguous(), vs.contiguous(), torch.arange(len(rows), device="cuda"), own, P)
            one = brq.paged_attention(layer.plan, qs[-1:].contiguous(), own, t,
                                      torch.tensor([len(rows)], dtype=torch.int32, device="cuda"), P)
            # the same sums of at most 27 keys; a query's rows may go another way through the kernels: 2^-20 of the norm
            assert (attended[b, leaf] - one[0]).norm() <= 2.0 ** -18 * one.norm()
            last = layer.after(x[b * N + leaf][None], attended[b, leaf][None], expert[b * N + leaf][None])
            assert (out[b * N + leaf] - last[0]).norm() <= 2.0 ** -18 * last.norm()

    # accept the path to draft 5 of either sample
    before = X.Cache.from_bytes(cache.cpu().numpy(), D, P)
    src, dst = torch.full((B, N), -1, device="cuda"), torch.full((B, N), -1, device="cuda")
    for b in range(B):
        path = [j for j in range(N) if masks[b][5] >> j & 1]
        src[b, :len(path)], dst[b, :len(path)] = slots[b, path], slots[b, :len(path)]
    brq.kv_move(cache, src.view(-1), dst.view(-1), D, P)
    X.move(before, src.view(-1).tolist(), dst.view(-1).tolist())
    assert np.array_equal(cache.cpu().numpy(), before.to_bytes())
    brq.kv_free(kids, refs), brq.kv_free(table, refs)
    assert not refs.any()


def inputs():
    import butterfly_rotation_quantization_amd as brq
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x, w = brq.mx_quantize(None, rand(300, 4096)), brq.mx_quantize(None, rand(512, 4096))
    experts = [z.view(2, 256, -1) for z in w]
    cache = brq.kv_cache(64, 2, 128, 64)
    kv = rand(400, 2, 128)
    brq.kv_append(None, kv, kv, torch.arange(400, device="cuda"), cache, 64)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    refs = torch.zeros(64, dtype=torch.int32, device="cuda")
    refs[:6] = 1
    q = rand(3, 4, 8, 128)
    mask = torch.from_numpy(to_mask([[1, 3, 5, 13]] * 3)).cuda()
    return dict(x=x, w=w, experts=experts, offsets=i32(0, 170, 300), bias=rand(512), res=rand(300, 512), cache=cache,
                table=table, refs=refs, lens=i32(70, 100, 3), q=q, mask=mask, src=torch.arange(600, device="cuda") % 128,
                dst=torch.arange(600, device="cuda") + 1024, parents=i32(0, 1, 1, 2))


def calls(i, stream):
    """Every call with nothing but its inputs given, temporaries and all."""
    import butterfly_rotation_quantization_amd as brq
    a = brq.mx_linear(*i["x"], *i["w"], bias=i["bias"], act="gelu", residual=i["res"], stream=stream)
    b = brq.mx_grouped_matmul(*i["x"], *i["experts"], i["offsets"], act="silu", stream=stream)
    c = brq.tree_attention(None, i["q"], i["cache"], i["table"], i["lens"], i["mask"], 64, stream=stream)
    kids, lens = brq.kv_fork(i["table"], i["lens"], i["parents"], i["refs"], stream=stream)
    slots = brq.kv_reserve(i["cache"], kids, lens, i["refs"], 70, 128, 64, stream=stream)
    brq.kv_move(i["cache"], i["src"], i["dst"], 128, 64, stream=stream)
    d = brq.tree_attention(None, i["q"][:1].repeat(4, 1, 1, 1) if stream is None else i["q4"], i["cache"], kids, lens,
                           i["mask4"], 64, stream=stream)
    return a, b, c, lens, slots, d, i["cache"]


def prepared():
    i = inputs()
    i["q4"], i["mask4"] = i["q"][:1].repeat(4, 1, 1, 1), i["mask"][:1].repeat(4, 1)
    return i


@pytest.mark.parametrize("raw", [False, True])
def test_temporaries_outlive_the_calls(raw):
    """The stream is busy while the host makes all the calls and the current stream overwrites all it is given."""
    import torch
    announce(f"step's calls on a busy stream raw={raw}")
    want = [t.clone() for t in calls(prepared(), None)]
    torch.cuda.synchronize()
    s, i = torch.cuda.Stream(), prepared()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = calls(i, s.cuda_stream if raw else s)
    junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
            for n in (300 * 512 * 2, 300 * 256 * 2, 3 * 4 * 8 * 128 * 4, 4 * 70 * 8, 1 << 16, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
    assert not s.query(), "the stream was to be busy still"
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and len(junk) == 32


def test_two_streams_at_once():
    """Calls of the same kinds ahead on two streams, each with workspaces and a cache of its own."""
    import torch
    announce("step's calls on two streams")
    want = [t.clone() for t in calls(prepared(), None)]
    pair, streams = (prepared(), prepared()), (torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    got = [calls(i, s) for i, s in zip(pair, streams)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_graphs_that_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn with other work between: nothing of one is left for the other."""
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("step's graphs sharing workspaces")
    i = prepared()
    ws = torch.zeros(max(brq.mx_matmul_workspace(300, 512, 4096).numel(),
                         brq.mx_grouped_matmul_workspace(300, 2, 256, 4096).numel(),
                         brq.tree_attention_workspace(3, 4, 8, 2, 128).numel()), dtype=torch.uint8, device="cuda")
    y, z, o = (torch.zeros(s, device="cuda") for s in ((300, 512), (300, 256), (3, 4, 8, 128)))
    steps = [lambda: brq.mx_linear(*i["x"], *i["w"], bias=i["bias"], act="gelu", residual=i["res"], y=y, ws=ws),
             lambda: brq.mx_grouped_matmul(*i["x"], *i["experts"], i["offsets"], act="silu", y=z, ws=ws),
             lambda: brq.tree_attention(None, i["q"], i["cache"], i["table"], i["lens"], i["mask"], 64, out=o, ws=ws)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for f in steps:
            f()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, z, o)]
    for f in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            f()
        graphs.append(g)
    for turn in range(4):
        for k in ((0, 1, 2), (2, 0, 1), (1, 2, 0), (0, 2, 1))[turn]:
            (y, z, o)[k].zero_()
            torch.cuda.synchronize()
            graphs[k].replay()
            torch.cuda.synchronize()
            assert torch.equal((y, z, o)[k], want[k]), (turn, k)

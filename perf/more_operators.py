"""Cases of the operators beside the microscaled 4-bit products, cache and
attention of one token: the product with an epilogue, products grouped by
expert, attention of a tree of drafted tokens over the paged cache, and the
moving, forking, reserving and freeing of the cache's tokens and pages.

``run`` computes each case in a plain form of elementary torch operations in
32 bits, or, with ``own`` set, through the package's entry points.  Both sides
take the same inputs, byte for byte.

Format.  A row is cut into blocks of 32 values that share a scale 2^e, stored
as the byte e + 127; a value is one of +-(0, 1/2, 1, 3/2, 2, 3, 4, 6) times it,
its 4-bit code (the sign in bit 3) in the low half of its byte for the even
value of a pair.

Cache.  [pages][key-value heads][bytes of one head's page] with, for a page of
P tokens and head dimension D: the keys' codes [P][D/2]; the values' codes
[P/4][16][4][D/32], which hold for each four tokens and each of 16 runs of
D/16 dimensions the four tokens' codes one after the other; the keys' scales
[P][D/32]; the values' scales [P/4][D/32][4].  Slot s is token s % P of page
s / P.

Epilogue.  y = act(a b^T + bias) * mul + residual, each part if given.

Tree.  Row (b, i) of the queries, with the bits of mask[b, i], sees the tokens
at positions below lens[b] and, for each set bit j, the one at lens[b] + j; with
a window, the last `window` of these.  A row whose mask is 0 is padding, its
output zero.

Pages.  refs counts the table rows that hold a page; a page with none is free.
A fork gives a child its parent's row.  A reservation gives a sequence, for each
of its next tokens, a page that no other row holds: in the order of sequences
and positions, the lowest free pages, with the first tokens of a shared page
copied (whole sixteens of them).  What counts as free or shared is what did when
the call began.
"""

import math
import random
from functools import reduce

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # Decode of one sequence: the down projection of an 11008-wide MLP, added to the residual stream.
        {"name": "linear 1x4096x11008", "op": "linear", "T": 1, "m": 4096, "n": 11008, "bias": False, "act": None,
         "mul": False, "residual": True, "out": "bf16"},
        # A prompt of 2048 tokens through a 70B-shaped up projection with bias and activation.
        {"name": "linear 2048x28672x8192", "op": "linear", "T": 2048, "m": 28672, "n": 8192, "bias": True,
         "act": "gelu", "mul": False, "residual": False, "out": "bf16"},
        # Decode of 16 tokens, two of 8 experts each: most experts see a few rows.
        {"name": "grouped 32x8x11008x4096", "op": "grouped", "T": 32, "E": 8, "m": 11008, "n": 4096, "skew": 0.7,
         "bias": False, "act": "silu", "mul": True, "residual": False, "out": "bf16"},
        # Many small experts, about 12 rows each, some with none.
        {"name": "grouped 777x64x1376x2048", "op": "grouped", "T": 777, "E": 64, "m": 1376, "n": 2048, "skew": 1.0,
         "bias": True, "act": "gelu_tanh", "mul": False, "residual": False, "out": "f32"},
        # A prompt of 4096 tokens, two of 8 experts each.
        {"name": "grouped 8192x8x4096x11008", "op": "grouped", "T": 8192, "E": 8, "m": 4096, "n": 11008, "skew": 0.4,
         "bias": False, "act": None, "mul": False, "residual": False, "out": "bf16"},
        # One conversation of a thousand tokens, a small tree: latency.
        {"name": "tree 1x7 of 1000", "op": "tree", "B": 1, "N": 7, "hq": 32, "hkv": 8, "D": 128, "page": 64,
         "short": 1000, "long": 1000, "window": 0, "rot": True, "dtype": "bf16"},
        # A serving batch: 32 sequences of 17 to 16384 tokens, eight drafted tokens each.
        {"name": "tree 32x8 of (17..16384)", "op": "tree", "B": 32, "N": 8, "hq": 64, "hkv": 8, "D": 128, "page": 32,
         "short": 17, "long": 16384, "window": 0, "rot": True, "dtype": "bf16"},
        # Four long documents with the largest trees.
        {"name": "tree 4x64 of 32768", "op": "tree", "B": 4, "N": 64, "hq": 64, "hkv": 8, "D": 128, "page": 128,
         "short": 32000, "long": 32768, "window": 0, "rot": False, "dtype": "f16"},
        # After such a step: the accepted drafts of 32 sequences move to the front of their trees.
        {"name": "move 32x5 accepted", "op": "move", "kind": "accept", "B": 32, "most": 5, "N": 16, "hkv": 8,
         "D": 128, "page": 32},
        # Half of a long sequence's tokens are kept, moved together into other pages.
        {"name": "move 30001 kept", "op": "move", "kind": "keep", "B": 1, "most": 30001, "N": 0, "hkv": 8, "D": 128,
         "page": 64},
        # 128 samples of 16 prompts: pages shared, the last one of each copied.
        {"name": "fork 16 to 128", "op": "fork", "B": 16, "F": 128, "short": 500, "long": 8000, "tokens": 8, "hkv": 8,
         "D": 128, "page": 64, "spare": 4096},
        # One prompt sampled twice.
        {"name": "fork 1 to 2", "op": "fork", "B": 1, "F": 2, "short": 333, "long": 333, "tokens": 1, "hkv": 8,
         "D": 128, "page": 16, "spare": 100},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "tree", "tree", "move", "fork"])
    if op in ("linear", "grouped"):
        act = rng.choice([None, "relu", "gelu", "gelu_tanh", "silu"])
        c = {"op": op, "bias": rng.random() < 0.5, "act": act, "mul": rng.random() < 0.4,
             "residual": rng.random() < 0.4, "out": rng.choice(["bf16", "f16", "f32"])}
        if op == "linear":
            c["n"] = BLOCK * (_log(rng, 256, 28672) // BLOCK)
            c["m"] = _log(rng, 128, 16384)
            c["T"] = _log(rng, 1, min(8192, 400_000_000_000 // (c["m"] * c["n"])))
            return c
        c["n"] = BLOCK * (_log(rng, 256, 11008) // BLOCK)
        c["m"] = _log(rng, 128, 11008)
        c["E"] = _log(rng, 2, min(256, 400_000_000 // (c["m"] * c["n"])))
        c["T"] = _log(rng, 1, min(16384, 400_000_000_000 // (c["m"] * c["n"])))
        c["skew"] = rng.choice([0.0, 0.4, 0.7, 1.0, 2.0])
        return c
    c = {"op": op, "hkv": rng.choice([1, 2, 4, 8, 16]), "D": rng.choice([64, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 128, 256])}
    if op == "tree":
        c["N"] = _log(rng, 1, 64)
        c["hq"] = c["hkv"] * rng.choice([1, 4, 5, 8, 16])
        c["B"] = _log(rng, 1, min(64, 1_000_000 // (c["N"] * c["hq"])))
        most = min(60_000_000_000 // (c["B"] * c["N"] * c["hq"] * c["D"]), 200_000_000 // (c["B"] * c["hkv"] * c["D"]))
        c["long"] = _log(rng, 16, min(131072, max(16, most // 2)))
        c["short"] = rng.choice([c["long"], max(1, c["long"] // 3), 0])
        c["window"] = rng.choice([0, 0, 0, 1000, 5])
        c["rot"] = rng.random() < 0.6
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        return c
    if op == "move":
        c["kind"] = rng.choice(["accept", "keep"])
        c["B"] = _log(rng, 1, 128)
        if c["kind"] == "accept":
            c["N"] = _log(rng, 2, 64)
            c["most"] = rng.randint(1, (c["N"] + 1) // 2)
        else:
            c["N"] = 0
            c["most"] = _log(rng, 16, max(16, 30_000_000 // (c["B"] * c["hkv"] * c["D"])))
        return c
    c["B"] = _log(rng, 1, 32)
    c["F"] = _log(rng, 1, min(256, max(1, 16_000_000 // (c["hkv"] * c["D"] * c["page"]))))
    c["long"] = _log(rng, 16, min(16384, max(16, 60_000_000 // (c["B"] * c["hkv"] * c["D"]))))
    c["short"] = rng.choice([c["long"], max(1, c["long"] // 3), 1])
    c["tokens"] = _log(rng, 1, 64)
    c["spare"] = c["F"] * (2 + (c["tokens"] - 1) // c["page"]) + _log(rng, 1, 500)
    return c


def _lens(c):
    """Sequence lengths from the shortest to the longest, evenly in their logarithm."""
    a, b, B = math.log(c["short"] + 1), math.log(c["long"] + 1), c["B"]
    return [int(round(math.exp(b if B == 1 else a + (b - a) * i / (B - 1)))) - 1 for i in range(B)]


def _counts(c):
    """Rows of each expert, the busiest first: shares fall as a power of the rank."""
    share = [(e + 1) ** -c["skew"] for e in range(c["E"])]
    at, ends = 0.0, []
    for s in share:
        at += s
        ends.append(int(round(c["T"] * at / sum(share))))
    return [b - a for a, b in zip([0] + ends, ends)]


def work(case):
    c, size = case, {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] in ("linear", "grouped"):
        weights = 1 if c["op"] == "linear" else sum(n > 0 for n in _counts(c))
        out = c["T"] * c["m"] * size[c["out"]]
        return {"bytes": (c["T"] + weights * c["m"]) * c["n"] * 17 / 32 + out * (1 + c["mul"] + c["residual"])
                + (weights * c["m"] * size[c["out"]] if c["bias"] else 0),
                "flops": 2 * c["T"] * c["m"] * c["n"]}
    token = c["hkv"] * c["D"] * 17 / 16  # bytes of a cached token
    if c["op"] == "tree":
        keys = [min(n, c["window"] or n) + c["N"] for n in _lens(c)]
        return {"bytes": sum(keys) * token + 2 * c["B"] * c["N"] * c["hq"] * c["D"] * size[c["dtype"]],
                "flops": 4 * sum(keys) * c["N"] * c["hq"] * c["D"]}
    if c["op"] == "move":
        tokens = c["B"] * (c["most"] + 1) / 2 if c["kind"] == "accept" else c["B"] * (c["most"] // 2)
        return {"bytes": 2 * tokens * token + 16 * c["B"] * c["most"], "flops": c["B"] * c["most"]}
    lens, P = _lens(c), c["page"]
    rows = [lens[f % c["B"]] for f in range(c["F"])]
    copied = sum(n % P for n in rows)
    entries = sum((n + P - 1) // P for n in rows)
    return {"bytes": 2 * copied * token + 8 * entries + 8 * c["F"] * c["tokens"] + 4 * (entries + c["spare"]),
            "flops": 2 * entries}


# ------------------------------------------------------------------ the inputs

def _dev():
    return torch.device("cuda")


def _activations(gen, rows, cols, dtype):
    """Normal values with every 128th channel or so an outlier channel, 20 times as large."""
    x = torch.randn((rows, cols), generator=gen, device=_dev())
    hot = torch.rand((cols,), generator=gen, device=_dev()) < 1 / 128
    return (x * torch.where(hot, 20.0, 1.0)).to(DTYPES[dtype])


def _weight(gen, rows, n):
    """Codes and scales of a weight whose rows differ in size up to twofold; products with activations are about 1."""
    w = torch.randn((rows, n), generator=gen, device=_dev()) / math.sqrt(2 * n)
    return _quantise(w * (1 + torch.rand((rows, 1), generator=gen, device=_dev())))


def _pages(gen, total, P, H, D):
    """A cache of `total` pages of quantised normal keys and values."""
    parts = []
    for _ in "kv":
        codes, scales = _quantise(torch.randn((total * P * H, D), generator=gen, device=_dev()))
        parts += [codes.view(total, P, H, -1), scales.view(total, P, H, -1)]
    return _lay_out(*parts)


def _table(gen, lens, P, W, total):
    """int32 [len(lens), W]: distinct random ones of `total` pages for each sequence's tokens, -1 behind them."""
    used = torch.arange(W, device=_dev()) < ((lens + P - 1) // P)[:, None]
    table = torch.full((len(lens), W), -1, device=_dev(), dtype=torch.int32)
    table[used] = torch.randperm(total, generator=gen, device=_dev())[: int(used.sum())].to(torch.int32)
    return table


def _tree(rng, N):
    """Ancestor bits of N drafted tokens of which at least half are there: each follows an earlier one or none."""
    masks, there = [], rng.randint((N + 1) // 2, N)
    for j in range(there):
        parent = rng.randint(max(-1, j - 6), j - 1)
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
    masks += [0] * (N - there)
    return [m - (1 << 64) if m >> 63 else m for m in masks]


def _accepted(rng, N, most):
    """(from, to) places of 1 to `most` accepted drafts: the first ones lie where they belong."""
    n = rng.randint(1, most)
    stay = rng.randint(0, n)
    return list(range(stay)) + sorted(rng.sample(range(n, N), min(n - stay, N - n))), n


def _epilogue(gen, c, s, groups):
    t, m = DTYPES[c["out"]], c["m"]
    new = lambda *shape: torch.randn(shape, generator=gen, device=_dev()).to(t)  # noqa: E731
    s["bias"] = (new(groups, m) if c["op"] == "grouped" else new(m)) if c["bias"] else None
    s["mul"] = new(c["T"], m) if c["mul"] else None
    s["residual"] = new(c["T"], m) if c["residual"] else None


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=_dev())
    gen.manual_seed(int(seed) * 7919 + 29)
    rng = random.Random(int(seed) * 104729 + 31)
    s = {"case": c, "plan": None, "signs": None, "ws": None}
    if own:
        import butterfly_rotation_quantization_amd as brq
    if c["op"] == "linear":
        s["a"] = _quantise(_activations(gen, c["T"], c["n"], "bf16"))
        s["b"] = _weight(gen, c["m"], c["n"])
        _epilogue(gen, c, s, 1)
        if own:
            s["ws"] = brq.mx_matmul_workspace(c["T"], c["m"], c["n"])
        return s
    if c["op"] == "grouped":
        s["a"] = _quantise(_activations(gen, c["T"], c["n"], "bf16"))
        E, m, n = c["E"], c["m"], c["n"]
        codes = torch.empty((E, m, n // 2), dtype=torch.uint8, device=_dev())
        scales = torch.empty((E, m, n // BLOCK), dtype=torch.uint8, device=_dev())
        for e in range(E):
            codes[e], scales[e] = _weight(gen, m, n)
        s["b"] = (codes, scales)
        s["counts"] = _counts(c)
        rng.shuffle(s["counts"])
        ends = reduce(lambda a, k: a + [a[-1] + k], s["counts"], [0])
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=_dev())
        _epilogue(gen, c, s, E)
        if own:
            s["ws"] = brq.mx_grouped_matmul_workspace(c["T"], E, m, n)
        return s
    P, D, H = c["page"], c["D"], c["hkv"]
    if c["op"] == "tree":
        B, N = c["B"], c["N"]
        lens = torch.tensor(_lens(c), device=_dev())[torch.randperm(B, generator=gen, device=_dev())]
        most = (c["long"] + N + P - 1) // P
        total = int(((lens + N + P - 1) // P).sum())
        s["table"] = _table(gen, lens + N, P, most, total)
        s["cache"] = _pages(gen, total, P, H, D)
        s["mask"] = torch.tensor([_tree(rng, N) for _ in range(B)], dtype=torch.int64, device=_dev())
        s["lens"] = lens.to(torch.int32)
        s["q"] = (1.5 * torch.randn((B, N, c["hq"], D), generator=gen, device=_dev())).to(DTYPES[c["dtype"]])
        if c["rot"]:
            s["signs"] = (torch.randint(0, 2, (D,), generator=gen, device=_dev()) * 2 - 1).to(torch.int8)
        if own:
            if c["rot"]:
                s["plan"] = brq.Plan(D, (2,) * (D.bit_length() - 1), "hadamard", None, s["signs"].cpu().numpy())
            s["ws"] = brq.tree_attention_workspace(B, N, c["hq"], H, D)
        return s
    if c["op"] == "move":
        if c["kind"] == "accept":
            per = (c["N"] + P - 1) // P + 1  # pages that a sequence's drafts may lie in
            total = c["B"] * per
            page = torch.randperm(total, generator=gen, device=_dev()).view(c["B"], per).tolist()
            pairs = []
            for b in range(c["B"]):
                first = rng.randrange(P)
                place = lambda j: page[b][(first + j) // P] * P + (first + j) % P  # noqa: B023, E731
                path, n = _accepted(rng, c["N"], c["most"])
                pairs += [(place(j), place(i)) for i, j in enumerate(path)]
                pairs += [(-1, -1)] * (c["most"] - len(path))
            s["src"], s["dst"] = torch.tensor(pairs, dtype=torch.int64, device=_dev()).t().contiguous()
        else:
            before, keep = (c["most"] + P - 1) // P, c["most"] // 2
            after = (keep + P - 1) // P
            total = c["B"] * (before + after)
            page = torch.randperm(total, generator=gen, device=_dev()).view(c["B"], -1)
            src, dst = [], []
            for b in range(c["B"]):
                at = torch.randperm(c["most"], generator=gen, device=_dev())[:keep].sort().values
                src.append(page[b][at // P] * P + at % P)
                i = torch.arange(keep, device=_dev())
                dst.append(page[b][before + i // P] * P + i % P)
            s["src"], s["dst"] = torch.cat(src), torch.cat(dst)
        s["cache"] = _pages(gen, total, P, H, D)
        if own:
            s["ws"] = brq.kv_move_workspace(len(s["src"]), H, D)
        return s
    lens = torch.tensor(_lens(c), device=_dev())
    most = (c["long"] + c["tokens"] + P - 1) // P
    used = int(((lens + P - 1) // P).sum())
    total = used + c["spare"]
    s["table"], s["lens"] = _table(gen, lens, P, most, total), lens.to(torch.int32)
    s["refs"] = torch.zeros((total,), dtype=torch.int32, device=_dev())
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    s["parents"] = (torch.randperm(c["F"], generator=gen, device=_dev()) % c["B"]).to(torch.int32)
    s["cache"] = _pages(gen, total, P, H, D)
    if own:
        s["ws"] = brq.kv_reserve_workspace(c["F"], c["tokens"], P, total)
    return s


# ------------------------------------------------------------------ the plain forms

def _rotate(x, signs, inverse=False):
    """The random-sign Walsh-Hadamard transform of every len(signs) values of a row, in 32 bits."""
    d = signs.numel()

    def stage(y, stride):
        p = y.view(-1, d // (2 * stride), 2, stride)
        return torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), dim=2)

    y = x.reshape(-1, d)
    y = y if inverse else y * signs.float()
    y = reduce(stage, [1 << i for i in range(d.bit_length() - 1)], y).reshape(-1, d)
    y = y * float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    return (y * signs.float() if inverse else y).view(x.shape)


def _quantise(x):
    """(codes uint8 [rows, n/2], scale bytes uint8 [rows, n/32]) of the rows of x."""
    rows, n = x.shape
    y = x.float().view(rows, n // BLOCK, BLOCK)
    top = y.abs().amax(dim=2)
    e = ((top.view(torch.int32) >> 23) - 129).clamp(-127, 127)
    e = torch.where(top > 0, e, -127)
    u = y * ((127 - e) << 23).view(torch.float32)[:, :, None]
    a = u.abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    a = a.clamp(max=6)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(u).to(torch.uint8) << 3)
    return (code[:, :, 0::2] | (code[:, :, 1::2] << 4)).reshape(rows, n // 2), (e + 127).to(torch.uint8)


def _pairs():
    """[256, 2]: the two values of a byte of codes."""
    one = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=_dev())
    one = torch.cat((one, -one))
    byte = torch.arange(256, device=_dev())
    return torch.stack((one[byte & 15], one[byte >> 4]), dim=1)


def _values(codes, scales):
    """The values of codes [..., n/2] with scale bytes [..., n/32], in 32 bits."""
    v = _pairs()[codes.to(torch.int32)].view(*scales.shape, BLOCK)
    w = scales.to(torch.int32)
    return (v * torch.where(w > 0, w << 23, 0x400000).view(torch.float32)[..., None]).flatten(-2)


def _lay_out(kc, ks, vc, vs):
    """Pages [pages, heads, bytes] of codes and scales given as [pages, P, heads, ...]."""
    n, P, H, half = kc.shape
    quad = vc.view(n, P // 4, 4, H, 16, half // 16).permute(0, 3, 1, 4, 2, 5)
    parts = (kc.transpose(1, 2), quad, ks.transpose(1, 2), vs.view(n, P // 4, 4, H, -1).permute(0, 3, 1, 4, 2))
    return torch.cat([p.reshape(n, H, -1) for p in parts], dim=2)


def _parts(pages, P, D):
    """Codes and scales (kc, ks, vc, vs), each [..., P, bytes], of pages [..., bytes]."""
    lead, c, e = pages.shape[:-1], P * D // 2, P * D // BLOCK
    kc, vc, ks, vs = pages.split((c, c, e, e), dim=-1)
    vc = vc.reshape(*lead, P // 4, 16, 4, D // 32).transpose(-3, -2).reshape(*lead, P, D // 2)
    vs = vs.reshape(*lead, P // 4, D // BLOCK, 4).transpose(-2, -1).reshape(*lead, P, D // BLOCK)
    return kc.reshape(*lead, P, D // 2), ks.reshape(*lead, P, D // BLOCK), vc, vs


def _act(x, act):
    """The activation in x's own precision."""
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    if act == "gelu_tanh":
        return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _finish(y, bias, act, mul, residual):
    """The epilogue of rows y in y's own precision."""
    y = y if bias is None else y + bias.to(y.dtype)
    y = _act(y, act)
    y = y if mul is None else y * mul.to(y.dtype)
    return y if residual is None else y + residual.to(y.dtype)


def _groups(s):
    """(rows, expert) of every expert that has some."""
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            yield slice(at, at + n), e
        at += n


def _run_linear(s):
    c = s["case"]
    y = _values(*s["a"]) @ _values(*s["b"]).t()
    return _finish(y, s["bias"], c["act"], s["mul"], s["residual"]).to(DTYPES[c["out"]])


def _run_grouped(s):
    c = s["case"]
    x, part = _values(*s["a"]), lambda t, i: None if t is None else t[i]  # noqa: E731
    y = torch.empty((c["T"], c["m"]), dtype=DTYPES[c["out"]], device=_dev())
    for r, e in _groups(s):
        acc = x[r] @ _values(s["b"][0][e], s["b"][1][e]).t()
        y[r] = _finish(acc, part(s["bias"], e), c["act"], part(s["mul"], r), part(s["residual"], r)).to(y.dtype)
    return y


def _seen(c, lens, mask, keys):
    """bool [B, N, keys]: which positions a row sees."""
    mask = mask[:, :, None]
    j = torch.arange(keys, device=_dev()) - lens.long()[:, None, None]  # the place among the drafts
    draft = j.clamp(0, 63)
    seen = torch.where(j < 0, mask != 0, (j < 64) & ((mask >> draft) & 1 == 1))
    if c["window"]:
        bits = (mask >> torch.arange(64, device=_dev())) & 1
        later = bits.flip(2).cumsum(2).flip(2)  # tokens seen from a draft on, itself among them
        behind = torch.where(j < 0, later[:, :, :1] - j, torch.gather(later, 2, draft.expand(seen.shape)))
        seen = seen & (behind <= c["window"])
    return seen


def _run_tree(s):
    c = s["case"]
    B, N, H, D, P = c["B"], c["N"], c["hkv"], c["D"], c["page"]
    q = s["q"].float()
    q = (_rotate(q, s["signs"]) if c["rot"] else q).view(B, N, H, -1, D).transpose(1, 2) / math.sqrt(D)
    G = q.shape[3]
    pages = s["cache"][s["table"].clamp(min=0).long()].transpose(1, 2)
    kc, ks, vc, vs = _parts(pages, P, D)
    del pages
    score = torch.matmul(q.reshape(B, H, N * G, D), _values(kc, ks).flatten(2, 3).transpose(2, 3))
    score = score.view(B, H, N, G, -1)
    seen = _seen(c, s["lens"], s["mask"], score.shape[4])
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(dim=4, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    del score
    total = p.sum(dim=4, keepdim=True)
    o = torch.matmul(p.view(B, H, N * G, -1), _values(vc, vs).flatten(2, 3)).view(B, H, N, G, D)
    o = (o / torch.where(total > 0, total, 1.0)).transpose(1, 2).reshape(B, N, -1, D)
    return (_rotate(o, s["signs"], inverse=True) if c["rot"] else o).to(DTYPES[c["dtype"]])


def _places(c, slots):
    """Byte positions in the flat cache of the tokens: [tokens, heads, bytes of a token]."""
    P, D, H = c["page"], c["D"], c["hkv"]
    lay = torch.cat(_parts(torch.arange(P * D * 17 // 16, device=_dev()), P, D), dim=1)
    base = (slots // P)[:, None] * H + torch.arange(H, device=_dev())
    return (base * (P * D * 17 // 16))[:, :, None] + lay[slots % P][:, None, :]


def _copy(c, cache, src, dst, ok):
    """The tokens of slots src to slots dst where ok; the others repeat the first of these."""
    k, flat = ok.int().argmax(), cache.view(-1)
    src, dst = (torch.where(ok, x, x[k]).clamp(min=0) for x in (src, dst))
    dst = torch.where(ok.any(), dst, src)
    flat[_places(c, dst)] = flat[_places(c, src)]


def _run_move(s):
    _copy(s["case"], s["cache"], s["src"], s["dst"], (s["src"] >= 0) & (s["dst"] >= 0))
    return s["cache"]


def _run_fork(s):
    """A fork of the parents' rows, a reservation for the children, and the children freed again."""
    c, refs, P = s["case"], s["refs"], s["case"]["page"]
    table = s["table"][s["parents"].long()]
    lens = s["lens"][s["parents"].long()].long()
    here = table >= 0
    refs += torch.zeros_like(refs).index_add_(0, table.clamp(min=0).flatten().long(), here.flatten().int())
    # the reservation: entries of pages from that of the first new token to that of the last
    F, W = table.shape
    at = torch.arange(W, device=_dev())
    wanted = (at >= (lens // P)[:, None]) & (at <= ((lens + c["tokens"] - 1) // P)[:, None])
    need = wanted & ~(here & (refs[table.clamp(min=0).long()] == 1))
    rank = need.flatten().long().cumsum(0).view(F, W) - 1
    free = torch.sort(refs > 0, stable=True).indices.to(torch.int32)
    room = need & (rank < (refs <= 0).sum())
    fresh = torch.where(room, free[rank.clamp(0, len(free) - 1)], table)
    # copies: the first tokens of the page that holds some
    first = (lens // P).clamp(max=W - 1)[:, None]
    old, new = table.gather(1, first)[:, 0], fresh.gather(1, first)[:, 0]
    count = torch.where((old != new) & (old >= 0), (lens % P + 15) // 16 * 16, 0)
    t = torch.arange(P, device=_dev())
    slot = lambda page: (page.long()[:, None] * P + t).flatten()  # noqa: E731
    _copy(c, s["cache"], slot(old), slot(new), (t < count[:, None]).flatten())
    moved = room & here
    refs -= torch.zeros_like(refs).index_add_(0, table.clamp(min=0).flatten().long(), moved.flatten().int())
    refs += torch.zeros_like(refs).index_add_(0, fresh.clamp(min=0).flatten().long(), room.flatten().int())
    pos = lens[:, None] + torch.arange(c["tokens"], device=_dev())
    slots = fresh.gather(1, pos // P).long() * P + pos % P
    # freed
    gone = (fresh >= 0).flatten().int()
    refs -= torch.zeros_like(refs).index_add_(0, fresh.clamp(min=0).flatten().long(), gone)
    return {"slots": slots, "lens": lens.to(torch.int32), "refs": refs, "cache": s["cache"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"linear": _run_linear, "grouped": _run_grouped, "tree": _run_tree, "move": _run_move,
                "fork": _run_fork}[c["op"]](s)
    import butterfly_rotation_quantization_amd as brq
    if c["op"] == "linear":
        return brq.mx_linear(*s["a"], *s["b"], bias=s["bias"], act=c["act"], mul=s["mul"], residual=s["residual"],
                             out_dtype=DTYPES[c["out"]], ws=s["ws"])
    if c["op"] == "grouped":
        return brq.mx_grouped_matmul(*s["a"], *s["b"], s["offsets"], bias=s["bias"], act=c["act"], mul=s["mul"],
                                     residual=s["residual"], out_dtype=DTYPES[c["out"]], ws=s["ws"])
    if c["op"] == "tree":
        return brq.tree_attention(s["plan"], s["q"], s["cache"], s["table"], s["lens"], s["mask"], c["page"],
                                  window=c["window"], ws=s["ws"])
    if c["op"] == "move":
        return brq.kv_move(s["cache"], s["src"], s["dst"], c["D"], c["page"], ws=s["ws"])
    table, lens = brq.kv_fork(s["table"], s["lens"], s["parents"], s["refs"])
    slots = brq.kv_reserve(s["cache"], table, lens, s["refs"], c["tokens"], c["D"], c["page"], ws=s["ws"])
    brq.kv_free(table, s["refs"])
    return {"slots": slots, "lens": lens, "refs": s["refs"], "cache": s["cache"]}


# ------------------------------------------------------------------ 64 bits

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode64(codes, scales):
    """Values of [..., bytes] codes and [..., bytes] scales."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=_dev())
    v = torch.stack((grid[(codes % 16).long()], grid[(codes // 16).long()]), dim=-1).flatten(-2)
    s = torch.pow(torch.full(scales.shape, 2.0, dtype=torch.float64, device=_dev()), scales.double() - 127)
    return v * s.repeat_interleave(BLOCK, dim=-1)


def _epilogue64(y, c, bias, mul, residual):
    if bias is not None:
        y = y + bias.double()
    if c["act"] == "relu":
        y = y.clamp(min=0)
    elif c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    if mul is not None:
        y = y * mul.double()
    return y if residual is None else y + residual.double()


def _hadamard64(d):
    """The orthonormal matrix: entry (i, j) is (-1)^popcount(i & j) / sqrt(d)."""
    i = torch.arange(d, device=_dev())
    both = i[:, None] & i[None, :]
    ones = torch.zeros_like(both)
    for b in range(d.bit_length()):
        ones += (both >> b) & 1
    return (1 - 2 * (ones % 2)).double() / math.sqrt(d)


def _fields(c, pages):
    """Views of pages [pages, heads, bytes]: keys' codes and scales by token, values' codes and scales by four."""
    P, D, (n, H, _) = c["page"], c["D"], pages.shape
    half, few = P * D // 2, P * D // 32
    cut = lambda a, w, *shape: pages[:, :, a : a + w].unflatten(2, shape)  # noqa: E731
    return (cut(0, half, P, D // 2), cut(2 * half, few, P, D // 32),
            cut(half, half, P // 4, 16, 4, D // 32), cut(2 * half + few, few, P // 4, D // 32, 4))


def _tree64(s, b):
    """Attention of the rows of sequence b over its pages one after the other, in 64 bits."""
    c = s["case"]
    N, H, D, P = c["N"], c["hkv"], c["D"], c["page"]
    n = int(s["lens"][b])
    pages = s["cache"][s["table"][b, : (n + N + P - 1) // P].long()]
    kc, ks, vc, vs = _fields(c, pages)
    k = _decode64(kc, ks)
    v = _decode64(vc.permute(0, 1, 2, 4, 3, 5).reshape(kc.shape), vs.permute(0, 1, 2, 4, 3).reshape(ks.shape))
    k, v = (x.transpose(0, 1).reshape(H, -1, D)[:, : n + N] for x in (k, v))
    seen = torch.zeros((N, n + N), dtype=torch.bool)
    for i, m in enumerate(s["mask"][b].tolist()):
        order = (list(range(n)) + [n + j for j in range(N) if m >> j & 1]) if m else []
        seen[i, order[-c["window"] :] if c["window"] else order] = True
    q = s["q"][b].double()
    m = _hadamard64(D) * s["signs"].double() if c["rot"] else None
    q = (q if m is None else q @ m.t()).view(N, H, -1, D).permute(1, 2, 0, 3)  # heads, heads of a group, rows
    score = torch.matmul(q, k[:, None].transpose(2, 3).contiguous()) / math.sqrt(D)
    score.masked_fill_(~seen.to(_dev()), -math.inf)
    p = torch.softmax(score, dim=3).nan_to_num_(nan=0.0)  # rows that see nothing
    o = torch.matmul(p, v[:, None]).permute(2, 0, 1, 3).reshape(N, -1, D)
    return o if m is None else o @ m


def _move64(c, cache, pairs):
    """The cache with the tokens of each pair of slots copied, all read first."""
    out = cache.clone()
    a, b = (torch.tensor(x, device=_dev(), dtype=torch.int64) for x in zip(*pairs))
    P = c["page"]
    for from_, to, quads in zip(_fields(c, cache), _fields(c, out), (False, False, True, True)):
        if not quads:
            to[b // P, :, b % P] = from_[a // P, :, a % P]
        else:
            to[b // P, :, b % P // 4, :, b % 4] = from_[a // P, :, a % P // 4, :, a % 4]
    return out


def _fork64(c, s):
    """The fork, the reservation and the freeing, one entry after the other."""
    P, table, refs = c["page"], s["table"].tolist(), s["refs"].tolist()
    rows = [list(table[p]) for p in s["parents"].tolist()]
    lens = [int(s["lens"][p]) for p in s["parents"].tolist()]
    for row in rows:
        for p in row:
            if p >= 0:
                refs[p] += 1
    free, held, pairs, slots = [p for p, r in enumerate(refs) if r == 0], list(refs), [], []
    for row, n in zip(rows, lens):
        for i in range(n // P, (n + c["tokens"] - 1) // P + 1):
            old = row[i]
            if old >= 0 and held[old] == 1:
                continue
            row[i] = free.pop(0)
            refs[row[i]] = 1
            if old >= 0:
                refs[old] -= 1
                if i == n // P:
                    pairs += [(old * P + t, row[i] * P + t) for t in range((n % P + 15) // 16 * 16)]
        slots.append([row[i // P] * P + i % P for i in range(n, n + c["tokens"])])
    for row in rows:
        for p in row:
            if p >= 0:
                refs[p] -= 1
    whole = lambda x, t: torch.tensor(x, dtype=t, device=_dev())  # noqa: E731
    return {"slots": whole(slots, torch.int64), "lens": whole(lens, torch.int32), "refs": whole(refs, torch.int32),
            "cache": _move64(c, s["cache"], pairs) if pairs else s["cache"]}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        return _epilogue64(_decode64(*s["a"]) @ _decode64(*s["b"]).t(), c, s["bias"], s["mul"], s["residual"])
    if c["op"] == "grouped":
        y = torch.empty((c["T"], c["m"]), dtype=torch.float64, device=_dev())
        first = 0
        for e, n in enumerate(s["counts"]):
            r, first = slice(first, first + n), first + n
            acc = _decode64(*(x[r] for x in s["a"])) @ _decode64(*(x[e] for x in s["b"])).t()
            y[r] = _epilogue64(acc, c, *(None if x is None else x[i] for x, i in
                                         ((s["bias"], e), (s["mul"], r), (s["residual"], r))))
        return y
    if c["op"] == "tree":
        return torch.stack([_tree64(s, b) for b in range(c["B"])])
    if c["op"] == "move":
        pairs = [(a, b) for a, b in zip(s["src"].tolist(), s["dst"].tolist()) if a >= 0]
        return _move64(c, s["cache"], pairs)
    return _fork64(c, s)

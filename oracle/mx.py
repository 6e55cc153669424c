"""Microscaled 4-bit rows, their product, the paged key-value cache and the
attention that reads it, from the definitions (include/brq.h), in float64 on
the CPU.  Only the transform ahead of the quantizer is in float32: its order of
additions is part of the definition, since a last bit can move a code."""

from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def hadamard32(x: np.ndarray, signs: np.ndarray | None, d: int) -> np.ndarray:
    """fl(1/sqrt d) H_d D on every d values of a row, in float32, the additions
    in the order of strides 1, 2, 4, ..., d/2."""
    y = np.asarray(x, dtype=np.float32).reshape(-1, d)
    if signs is not None:
        y = y * np.asarray(signs, dtype=np.float32)
    s = 1
    while s < d:
        p = y.reshape(-1, d // (2 * s), 2, s)
        y = np.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), axis=2).reshape(-1, d)
        s *= 2
    return (y * np.float32(1.0 / np.sqrt(d))).reshape(np.shape(x))


def hadamard64(d: int, signs: np.ndarray | None) -> np.ndarray:
    """The transform M = H_d D / sqrt(d) as a dense matrix."""
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(d) * (1.0 if signs is None else np.asarray(signs, dtype=np.float64))


def quantize(x: np.ndarray):
    """(codes uint8 [rows, n/2], scales uint8 [rows, n/32]) of float32 rows."""
    rows, n = x.shape
    v = np.asarray(x, dtype=np.float32).astype(np.float64).reshape(rows, n // BLOCK, BLOCK)
    top = np.abs(v).max(axis=2)
    bad = ~np.isfinite(v).all(axis=2)
    with np.errstate(divide="ignore"):
        e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1 - 2  # floor(log2) - 2
    e = np.where(top == 0, -127, np.clip(e, -127, 127))
    e = np.where(bad, 0, e)
    u = np.where(bad[..., None], 0.0, v) / np.ldexp(1.0, e)[..., None]
    mag = np.minimum(np.abs(u), 6.0)
    # distance to every magnitude; of two at the same distance the even code
    dist = np.abs(mag[..., None] - MAGNITUDES)
    near = dist == dist.min(axis=-1, keepdims=True)
    code = np.where(near[..., ::2].any(axis=-1), 2 * near[..., ::2].argmax(axis=-1), near.argmax(axis=-1))
    neg = np.signbit(np.asarray(x, dtype=np.float32)).reshape(code.shape) & ~bad[..., None]
    code = (code + 8 * neg).astype(np.uint8).reshape(rows, n)
    return code[:, 0::2] | code[:, 1::2] << 4, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values [..., n] that codes [..., n/2] and scales [..., n/32] stand for."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = MAGNITUDES[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def matmul(a_codes, a_scales, b_codes, b_scales) -> np.ndarray:
    return values(a_codes, a_scales) @ values(b_codes, b_scales).T


# ------------------------------------------------------------------ paged cache

class Cache:
    """One key-value cache as codes and scales by page, head and token."""

    def __init__(self, pages, heads, D, P):
        self.shape = (pages, heads, P)
        self.D, self.P = D, P
        self.kc = np.zeros((pages, heads, P, D // 2), np.uint8)
        self.vc = np.zeros_like(self.kc)
        self.ks = np.zeros((pages, heads, P, D // BLOCK), np.uint8)
        self.vs = np.zeros_like(self.ks)

    @classmethod
    def from_bytes(cls, raw: np.ndarray, D: int, P: int) -> "Cache":
        pages, heads, _ = raw.shape
        self = cls(pages, heads, D, P)
        half, few = P * D // 2, P * D // BLOCK
        cut = np.split(raw, (half, 2 * half, 2 * half + few), axis=2)
        self.kc = cut[0].reshape(pages, heads, P, D // 2)
        v = cut[1].reshape(pages, heads, P // 4, 16, 4, D // 32)
        self.vc = v.transpose(0, 1, 2, 4, 3, 5).reshape(pages, heads, P, D // 2)
        self.ks = cut[2].reshape(pages, heads, P, D // BLOCK)
        s = cut[3].reshape(pages, heads, P // 4, D // BLOCK, 4)
        self.vs = s.transpose(0, 1, 2, 4, 3).reshape(pages, heads, P, D // BLOCK)
        return self

    def to_bytes(self) -> np.ndarray:
        pages, heads, P = self.shape
        D = self.D
        v = self.vc.reshape(pages, heads, P // 4, 4, 16, D // 32).transpose(0, 1, 2, 4, 3, 5)
        s = self.vs.reshape(pages, heads, P // 4, 4, D // BLOCK).transpose(0, 1, 2, 4, 3)
        return np.concatenate([np.ascontiguousarray(x).reshape(pages, heads, -1)
                               for x in (self.kc, v, self.ks, s)], axis=2)

    def append(self, k, v, slots, signs=None, rotate=False):
        """k, v float32 [tokens, heads, D]; slots outside the cache are skipped."""
        for x, codes, scales in ((k, self.kc, self.ks), (v, self.vc, self.vs)):
            y = hadamard32(x, signs, self.D) if rotate else np.asarray(x, np.float32)
            c, s = quantize(y.reshape(-1, self.D))
            c, s = (z.reshape(*y.shape[:2], -1) for z in (c, s))
            for i, slot in enumerate(slots):
                if 0 <= slot < self.shape[0] * self.P:
                    codes[slot // self.P, :, slot % self.P] = c[i]
                    scales[slot // self.P, :, slot % self.P] = s[i]

    def keys_values(self):
        """(k, v) [pages, heads, P, D] in float64, as stored (rotated)."""
        return values(self.kc, self.ks), values(self.vc, self.vs)


def attention(q, cache: Cache, table, lens, scale, window=0, M=None):
    """(out, lse, slack) of one token per sequence: q float64 [batch, q_heads,
    D]; M the dense transform the cache was appended with, or None.  slack is
    what the tests scale an error bound with: per output the sum of
    probabilities times magnitudes, and per head the largest sum of |q_i k_i|."""
    B, hq, D = q.shape
    pages, heads, P = cache.shape
    K, V = cache.keys_values()
    out, lse = np.zeros((B, hq, D)), np.full((B, hq), -np.inf)
    spread, terms = np.zeros((B, hq, D)), np.zeros((B, hq))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * P)
        keys = [(int(table[b, j // P]), j % P) for j in range(max(0, n - window) if window else 0, n)]
        keys = [(p, t) for p, t in keys if 0 <= p < pages]
        if not keys:
            continue
        at = tuple(np.array(x) for x in zip(*keys))
        for i in range(hq):
            h = i // (hq // heads)
            k, v = K[at[0], h, at[1]], V[at[0], h, at[1]]
            x = q[b, i] if M is None else M @ q[b, i]
            s = scale * (k @ x)
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            o, w = p @ v / total, p @ np.abs(v) / total
            out[b, i] = o if M is None else M.T @ o
            spread[b, i] = w if M is None else np.abs(M.T) @ w
            lse[b, i] = top + np.log(total)
            terms[b, i] = abs(scale) * (np.abs(k) @ np.abs(x)).max()
    return out, lse, (spread, terms)


# ------------------------------------------------------------------ epilogue of a product

def _erfc(z):
    from scipy.special import erfc
    return erfc(z)


def activation(x: np.ndarray, act):
    """(act(x), bound of a float32 evaluation's error in units of 2^-24): a
    probability of tail z = x / sqrt 2 or of logit g is off by the rounding of
    its argument times the logarithm's derivative (2 z, 1) besides a few units of its own."""
    one = np.ones_like(x)
    with np.errstate(over="ignore", invalid="ignore"):
        if act is None:
            return x, 0 * one
        if act == "relu":
            return np.where(x < 0, 0.0, x), 0 * one
        if act == "gelu":
            y = 0.5 * x * _erfc(-x / np.sqrt(2))
            return y, np.abs(y) * (20 + 4 * np.minimum(x, 0) ** 2) + 1e-30
        g = x if act == "silu" else np.sqrt(8 / np.pi) * (x + 0.044715 * x ** 3)
        y = np.where(g < -700, 0.0, x / (1 + np.exp(-np.maximum(g, -700))))
        return y, np.abs(y) * (12 + 6 * np.abs(np.minimum(g, 0))) + 1e-30


def epilogue(s: np.ndarray, bias=None, act=None, mul=None, residual=None):
    """(act(s + bias) * mul + residual, bound of the error of a float32
    evaluation from exact sums s, before the output's own rounding)."""
    half = 2.0 ** -24
    x = s if bias is None else s + bias
    err = 0 * x if bias is None else half * np.abs(x)
    y, own = activation(x, act)
    slope = 1.0 if act in (None, "relu") else 1.2  # the largest of any activation
    err = slope * err + half * own
    if mul is not None:
        y = y * mul
        err = err * np.abs(mul) + half * np.abs(y)
    if residual is not None:
        y = y + residual
        err = err + half * np.abs(y)
    return y, err


# ------------------------------------------------------------------ trees of drafts; tokens and pages moved and shared

def tree_attention(q, cache: Cache, table, lens, mask, scale, window=0, M=None):
    """attention() for q [batch, drafts, q_heads, D]: row i of sequence b sees the
    positions below lens[b] and lens[b] + j for the bits j of mask[b, i], of these the
    last `window`; nothing if mask[b, i] is 0 or lens[b] negative."""
    B, N, hq, D = q.shape
    pages, heads, P = cache.shape
    K, V = cache.keys_values()
    out, lse = np.zeros(q.shape), np.full((B, N, hq), -np.inf)
    spread, terms = np.zeros(q.shape), np.zeros((B, N, hq))
    for b in range(B):
        n = int(lens[b])
        for i in range(N):
            m = int(mask[b, i]) & (2 ** N - 1)
            if n < 0 or m == 0:
                continue
            at = np.concatenate((np.arange(min(n, table.shape[1] * P)), [n + j for j in range(64) if m >> j & 1])).astype(int)
            if window:
                first = n + bin(m).count("1") - window  # how many positions are passed over
                drafts = at[at >= n]
                at = np.concatenate((at[(at < n) & (at >= first)], drafts[max(0, len(drafts) - window):]))
            at = at[at < table.shape[1] * P]
            page = table[b, at // P]
            at, page = at[(page >= 0) & (page < pages)], page[(page >= 0) & (page < pages)]
            if not len(at):
                continue
            g = hq // heads
            x = q[b, i] if M is None else q[b, i] @ M.T
            for h in range(heads):
                k, v, xh = K[page, h, at % P], V[page, h, at % P], x[h * g:(h + 1) * g]
                s = scale * (xh @ k.T)
                top = s.max(1, keepdims=True)
                p = np.exp(s - top)
                total = p.sum(1, keepdims=True)
                o, w = p @ v / total, p @ np.abs(v) / total
                r = slice(h * g, (h + 1) * g)
                out[b, i, r] = o if M is None else o @ M
                spread[b, i, r] = w if M is None else w @ np.abs(M)
                lse[b, i, r] = (top + np.log(total))[:, 0]
                terms[b, i, r] = abs(scale) * (np.abs(xh) @ np.abs(k).T).max(1)
    return out, lse, (spread, terms)


def move(cache: Cache, src, dst):
    """Tokens of slots src to slots dst, all read first; pairs outside the cache skipped."""
    pages, _, P = cache.shape
    pairs = [(int(a), int(b)) for a, b in zip(src, dst) if 0 <= a < pages * P and 0 <= b < pages * P]
    for x in (cache.kc, cache.ks, cache.vc, cache.vs):
        old = x.copy()
        for a, b in pairs:
            x[b // P, :, b % P] = old[a // P, :, a % P]


def fork(table, lens, parents, refs):
    """(table, lens) of the children; refs updated."""
    out, n = np.full((len(parents), table.shape[1]), -1, np.int32), np.zeros(len(parents), np.int32)
    for f, p in enumerate(parents):
        if 0 <= p < len(table):
            n[f] = lens[p]
            for c, page in enumerate(table[p]):
                if 0 <= page < len(refs):
                    out[f, c] = page
                    refs[page] += 1
    return out, n


def reserve(cache: Cache, table, lens, refs, tokens):
    """Slots [batch, tokens] of the next tokens; cache, table and refs updated."""
    pages, _, P = cache.shape
    before = refs.copy()
    free = [p for p in range(pages) if before[p] <= 0]
    slots = np.full((len(lens), tokens), -1, np.int64)
    src, dst = [], []
    for b, n in enumerate(int(x) for x in lens):
        if n < 0:
            continue
        for c in range(n // P, min(table.shape[1], (n + tokens - 1) // P + 1)):
            old = int(table[b, c])
            holders = before[old] if 0 <= old < pages else 0  # below 1: a page that is free, whatever the entry says
            page = old
            if holders != 1:
                if not free:
                    continue
                page = free.pop(0)
                table[b, c] = page
                refs[page] = 1
                if holders > 1:
                    refs[old] -= 1
                    if c == n // P:
                        used = (n % P + 15) // 16 * 16
                        src += [old * P + t for t in range(used)]
                        dst += [page * P + t for t in range(used)]
            for t in range(max(n, c * P), min(n + tokens, (c + 1) * P)):
                slots[b, t - n] = page * P + t % P
    move(cache, src, dst)
    return slots


def free(table, refs, rows):
    for r in rows:
        if 0 <= r < len(table):
            for c, page in enumerate(table[r]):
                if 0 <= page < len(refs):
                    refs[page] -= 1
                table[r, c] = -1

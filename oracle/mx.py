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

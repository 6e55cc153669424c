"""Pins of the microscaled 4-bit oracle: the rounding against hand-worked
values, the transform against the dense matrix, and the cache layout."""

import numpy as np
import pytest

from oracle import mx as X


def one_block(vals):
    x = np.zeros((1, 32), np.float32)
    x[0, :len(vals)] = vals
    c, s = X.quantize(x)
    return X.values(c, s)[0, :len(vals)], int(s[0, 0])


def test_ties_go_to_the_even_code_and_large_values_saturate():
    got, s = one_block([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, -0.25, 0.2500001, 6.9, -7.9])
    assert s == 127
    assert got.tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -4.0, -0.0, 0.5, 6.0, -6.0]


@pytest.mark.parametrize("top,byte", [(1.0, 125), (1.999, 125), (2.0, 126), (2.0 ** 127, 252), (2.0 ** -125, 0),
                                      (2.0 ** -124, 1), (2.0 ** -140, 0), (0.0, 0), (np.inf, 255), (np.nan, 255)])
def test_scale_bytes(top, byte):
    assert one_block([top, 0.0])[1] == byte


def test_a_block_with_a_nan_stands_for_nan_and_leaves_its_neighbour():
    x = np.ones((1, 64), np.float32)
    x[0, 40] = np.nan
    v = X.values(*X.quantize(x))
    assert np.array_equal(v[0, :32], np.ones(32)) and np.isnan(v[0, 32:]).all()


def test_every_code_survives_a_round_trip():
    codes = np.arange(256, dtype=np.uint8).reshape(1, 256).repeat(16, axis=1)[:, :2048]
    scales = np.full((1, 128), 130, np.uint8)
    codes[:, ::16] = 0x77  # every block reaches 6, so its scale comes back
    v = X.values(codes, scales).astype(np.float32)
    c, s = X.quantize(v)
    assert np.array_equal(s, scales) and np.array_equal(X.values(c, s), v.astype(np.float64))
    assert np.array_equal(c, codes)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_fast_transform_is_the_dense_matrix(d):
    rng = np.random.default_rng(d)
    signs = rng.choice([-1.0, 1.0], d)
    M = X.hadamard64(d, signs)
    assert np.allclose(M @ M.T, np.eye(d), atol=1e-12)
    x = rng.standard_normal((5, 2 * d)).astype(np.float32)
    want = (x.astype(np.float64).reshape(-1, d) @ M.T).reshape(x.shape)
    # log2(d) additions and one product, each within 2^-24 of its result
    bound = (np.log2(d) + 2) * 2.0 ** -24 * np.sqrt(d) * np.abs(x).max()
    assert np.abs(X.hadamard32(x, signs, d) - want).max() <= bound


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 32)])
def test_cache_layout_round_trip(D, P):
    rng = np.random.default_rng(D)
    raw = rng.integers(0, 256, (3, 2, P * (D + D // 16)), dtype=np.int64).astype(np.uint8)
    assert np.array_equal(X.Cache.from_bytes(raw, D, P).to_bytes(), raw)
    # the first four tokens' first run of values' codes follow one another
    c = X.Cache.from_bytes(raw, D, P)
    w = D // 32
    assert np.array_equal(raw[1, 1, P * D // 2:P * D // 2 + 4 * w].reshape(4, w), c.vc[1, 1, :4, :w])


def test_attention_is_the_softmax_average():
    rng = np.random.default_rng(5)
    D, P = 64, 16
    cache = X.Cache(3, 1, D, P)
    k, v = rng.standard_normal((2, 20, 1, D)).astype(np.float32)
    table = np.array([[2, 0]])
    cache.append(k, v, [2 * P + j if j < P else j - P for j in range(20)])
    q = rng.standard_normal((1, 2, D))
    out, lse, _ = X.attention(q, cache, table, [20], 0.125)
    kk = X.values(*X.quantize(k[:, 0]))
    vv = X.values(*X.quantize(v[:, 0]))
    s = 0.125 * q[0] @ kk.T
    assert np.allclose(out[0], np.exp(s) @ vv / np.exp(s).sum(1, keepdims=True), atol=1e-12)
    assert np.allclose(lse[0], np.log(np.exp(s).sum(1)), atol=1e-12)
    out, lse, _ = X.attention(q, cache, table, [0], 0.125)
    assert not out.any() and np.isneginf(lse).all()

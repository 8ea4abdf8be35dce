"""The fp64 forms of the row operators against brute force and differences."""
import numpy as np
import pytest

from oracle import rows_oracle as R


def test_group_is_stable_and_drops():
    ids = np.array([[2, 0], [1, -1], [0, 7], [2, 2]], np.int32)
    counts, offsets, src, pos = R.group(ids, 3)
    assert counts.tolist() == [2, 1, 3] and offsets.tolist() == [0, 2, 3, 6]
    assert src.tolist() == [1, 4, 2, 0, 6, 7, -1, -1]
    assert pos.tolist() == [[3, 0], [2, -1], [1, -1], [4, 5]]


@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_against_differences(weighted):
    rng = np.random.default_rng(3)
    N, K, E, d = 5, 3, 4, 6
    ids = rng.integers(-1, E + 1, (N, K))
    _, offsets, src, pos = R.group(ids, E)
    w = rng.standard_normal((N, K)) if weighted else None
    rows, base, dy = rng.standard_normal((N * K, d)), rng.standard_normal((N, d)), rng.standard_normal((N, d))
    drows, dw, _ = R.unpermute_backward(dy, pos, w, rows, np.zeros((N * K, d)))

    def loss(rows_, w_):
        return float(np.sum(dy * R.unpermute(rows_, pos, w_, base)[0]))
    h = 1e-6
    for i in range(N * K):
        for j in range(d):
            up, dn = rows.copy(), rows.copy()
            up[i, j] += h
            dn[i, j] -= h
            assert abs((loss(up, w) - loss(dn, w)) / (2 * h) - drows[i, j]) < 1e-7
    if weighted:
        for t in range(N):
            for k in range(K):
                up, dn = w.copy(), w.copy()
                up[t, k] += h
                dn[t, k] -= h
                assert abs((loss(rows, up) - loss(rows, dn)) / (2 * h) - dw[t, k]) < 1e-7


def test_permute_gradient_against_differences():
    rng = np.random.default_rng(4)
    N, K, E, d = 4, 2, 3, 5
    _, _, src, pos = R.group(rng.integers(0, E + 1, (N, K)), E)
    x, g = rng.standard_normal((N, d)), rng.standard_normal((N * K, d))
    dx, _ = R.unpermute(g, pos)
    h = 1e-6
    for t in range(N):
        for j in range(d):
            up, dn = x.copy(), x.copy()
            up[t, j] += h
            dn[t, j] -= h
            z = np.zeros((N * K, d))
            num = np.sum(g * (R.permute(up, src, K, z) - R.permute(dn, src, K, z))) / (2 * h)
            assert abs(num - dx[t, j]) < 1e-7


def bf16_values(limit):
    """All finite positive bf16 patterns up to `limit`, as fp64."""
    bits = np.arange(1, 0x7F80, dtype=np.uint32) << 16
    v = bits.view(np.float32).astype(np.float64)
    return v[v <= limit]


def test_corrected_product_gives_the_quotients_integer():
    """For every significand of the largest value and every smaller bf16 value:
    q = x y, q + (x - s q) y with y = 1 / s rounded gives the integer of the
    rounded quotient x / s (half of the largest value is a tie but for the
    rounding of s, so the product alone does not).  Powers of two only shift
    both."""
    alone = 0
    for sig in range(128, 256):
        top = float(sig) / 128.0
        x = bf16_values(top)
        x = x[x > top / 1024.0].astype(np.float32)
        s = np.float32(top) * (np.float32(1.0) / np.float32(127.0))
        y = np.float32(1.0) / s
        q = x * y
        r = (x.astype(np.float64) - s.astype(np.float64) * q.astype(np.float64)).astype(np.float32)
        q1 = (r.astype(np.float64) * y.astype(np.float64) + q.astype(np.float64)).astype(np.float32)
        assert np.array_equal(np.rint(q1), np.rint(x / s)), sig
        alone += int(np.sum(np.rint(q) != np.rint(x / s)))
    assert alone > 0


def test_int8_product_against_floats():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((7, 48)), rng.standard_normal((5, 48))
    q, s = R.int8_quantize(x)
    c, t = R.int8_quantize(w)
    y = R.int8_product(q, s, c, t)
    # every operand is off by half a step of its row at most
    bound = 24.5 * (np.abs(x).max(1)[:, None] / 127 * np.abs(w).max(1)[None, :]) * 2 + \
        48 * s[:, None] * t[None, :]
    assert np.all(np.abs(y - x @ w.T) <= bound)

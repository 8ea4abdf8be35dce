"""Plain fp64 forms of the operators that take the layer apart (test
infrastructure): grouping, rows to the experts and back with their gradients,
rows kept in E4M3, and the 8-bit integer products.  Loops over the definitions,
nothing of the package."""
import numpy as np

E4M3_MAX = 448.0


def group(ids, E):
    """counts, offsets, sorted_src, src_pos of ids [N, K]; ids outside [0, E)
    have no place."""
    flat = np.asarray(ids).reshape(-1)
    order = [p for e in range(E) for p in np.flatnonzero(flat == e)]
    counts = np.array([np.sum(flat == e) for e in range(E)], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = np.full(flat.size, -1, np.int32)
    src[:len(order)] = order
    pos = np.full(flat.size, -1, np.int32)
    pos[order] = np.arange(len(order))
    return counts, offsets, src, pos.reshape(np.shape(ids))


def permute(x, src, K, out):
    """Sorted rows; behind them what out holds."""
    rows = np.array(out, np.float64)
    for r, p in enumerate(src):
        if p >= 0:
            rows[r] = x[p // K]
    return rows


def unpermute(rows, pos, weights=None, base=None):
    """y, and the sum of the absolute terms."""
    N, K = pos.shape
    y = np.zeros((N, rows.shape[1])) if base is None else np.array(base, np.float64)
    mag = np.abs(y)
    for t in range(N):
        for k in range(K):
            if pos[t, k] >= 0:
                term = rows[pos[t, k]] * (1.0 if weights is None else weights[t, k])
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def unpermute_backward(dy, pos, weights, rows, out):
    """grad_rows, grad_weights and the sums of the absolute products behind the
    latter."""
    N, K = pos.shape
    drows = np.array(out, np.float64)
    dw, mag = np.zeros((N, K)), np.zeros((N, K))
    for t in range(N):
        for k in range(K):
            p = pos[t, k]
            if p >= 0:
                drows[p] = dy[t] * (1.0 if weights is None else weights[t, k])
                if rows is not None:
                    dw[t, k] = np.dot(dy[t], rows[p])
                    mag[t, k] = np.dot(np.abs(dy[t]), np.abs(rows[p]))
    return drows, dw, mag


def int8_quantize(x):
    """Integers and scales of the rows of x (bf16 values in fp64): s = amax times
    1 / 127 and x / s, each rounded to fp32, the latter then to the nearest integer,
    halves to even."""
    x = np.asarray(x, np.float64).astype(np.float32)
    s = np.abs(x).max(axis=-1) * (np.float32(1.0) / np.float32(127.0))
    live = (s > 0)[..., None]
    q = np.where(live, np.rint(x / np.where(live, s[..., None], np.float32(1.0))), 0.0)
    return np.clip(q, -127, 127).astype(np.int8), s


def int8_product(q, s, w, ws):
    """q [n, k], w [cols, k] integers: the scaled product."""
    acc = q.astype(np.int64) @ w.astype(np.int64).T
    return acc.astype(np.float64) * s.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))

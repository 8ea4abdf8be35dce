"""Plain fp64 forms of the operators around the layer: the residual norm with
its gradients and the balance loss with its gradient.  NumPy only, written from
the formulas; used by the tests."""
import numpy as np


def rms_norm(x, w, eps, residual=None, post_w=None):
    """(r, y, a): r = residual + (post_w ? post_w x / rms(x) : x), y = w r a,
    a = 1 / rms(r), row by row."""
    x = x.astype(np.float64)
    u = x
    if post_w is not None:
        u = x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * post_w.astype(np.float64)
    r = u if residual is None else u + residual.astype(np.float64)
    a = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    return r, r * a * w.astype(np.float64), a


def rms_norm_backward(dy, r, w, eps, dres=None, x=None, post_w=None):
    """Gradients (dx, dr, dw, dw_post) at the stored r (and x)."""
    dy, r, w = (t.astype(np.float64) for t in (dy, r, w))
    a = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    n, h = r * a, dy * w
    dr = a * (h - n * np.mean(h * n, axis=1, keepdims=True))
    if dres is not None:
        dr = dr + dres.astype(np.float64)
    dw = np.sum(dy * n, axis=0)
    if post_w is None:
        return dr, dr, dw, None
    x = x.astype(np.float64)
    b = 1.0 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
    m, k = x * b, dr * post_w.astype(np.float64)
    return b * (k - m * np.mean(k * m, axis=1, keepdims=True)), dr, dw, np.sum(dr * m, axis=0)


def balance_scores(z, score):
    z = z.astype(np.float64)
    if score == "softmax":
        e = np.exp(z - z.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)
    s = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))),
                 np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    return s / s.sum(axis=1, keepdims=True) if score == "sigmoid_norm" else s


def segment_counts(ids, E, spans):
    out = np.zeros((len(spans), E), np.int64)
    for g, (lo, hi) in enumerate(spans):
        sel = ids[lo:hi].reshape(-1)
        sel = sel[(sel >= 0) & (sel < E)]
        out[g] = np.bincount(sel, minlength=E)
    return out


def balance_loss(z, counts, coef, score, spans):
    """(loss, mean scores [G, E]) with the given loads."""
    G, E = counts.shape
    mean = np.zeros((G, E))
    total = 0.0
    for g, (lo, hi) in enumerate(spans):
        if hi <= lo:
            continue
        mean[g] = balance_scores(z[lo:hi], score).mean(axis=0)
        c = counts[g].astype(np.float64)
        if c.sum() > 0:
            total += E * float(c @ mean[g]) / c.sum()
    return coef * total / G, mean


def balance_loss_backward(z, counts, coef, score, spans):
    """d loss / d z [N, E], and for every element the size of the terms that it
    is the difference of (for tolerances)."""
    G, E = counts.shape
    dz = np.zeros(z.shape)
    size = np.zeros(z.shape)
    for g, (lo, hi) in enumerate(spans):
        c = counts[g].astype(np.float64)
        if hi <= lo or c.sum() <= 0:
            continue
        f = E * c / c.sum()
        w = coef / G / (hi - lo)
        zz = z[lo:hi].astype(np.float64)
        p = balance_scores(zz, score)
        if score == "sigmoid":
            slope, along = p * balance_scores(-zz, "sigmoid"), np.zeros((hi - lo, 1))
        else:
            along = (p * f).sum(axis=1, keepdims=True)
            slope = p if score == "softmax" else p * balance_scores(-zz, "sigmoid")
        dz[lo:hi] = w * slope * (f - along)
        size[lo:hi] = w * slope * (f + along)
    return dz, size

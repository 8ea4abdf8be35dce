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
    if score == "sigmoid_norm":
        # log sigma relative to the row's largest, so that no row's sum is zero
        log = np.minimum(z, 0.0) - np.log1p(np.exp(-np.abs(z)))
        e = np.exp(log - log.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)
    return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))),
                    np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


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


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def expert_backward(x, dy, s, wg, wu, wd):
    """Gradients of sum_t dy_t . s_t (silu(x Wg^T) * (x Wu^T)) Wd^T for the rows
    of one expert, and the sizes of the terms they are sums of.  Returns a dict:
    dx, ds, wg, wu, wd, and under "mag" the same keys with every product's
    operands replaced by their absolute values."""
    x, dy, wg, wu, wd = (t.astype(np.float64) for t in (x, dy, wg, wu, wd))
    s = s.astype(np.float64)[:, None]
    G, U, Q = x @ wg.T, x @ wu.T, dy @ wd
    sg = _sigmoid(G)
    H = G * sg * U
    dU, dG = s * Q * G * sg, s * Q * U * sg * (1 + G * (1 - sg))
    out = dict(dx=dG @ wg + dU @ wu, ds=(Q * H).sum(1), wg=dG.T @ x, wu=dU.T @ x, wd=dy.T @ (s * H))
    aG, aU, aQ = np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T, np.abs(dy) @ np.abs(wd)
    out["mag"] = dict(dx=np.abs(dG) @ np.abs(wg) + np.abs(dU) @ np.abs(wu),
                      # dQ H + Q dH for relative errors of Q, G and U taken as one
                      ds=(aQ * np.abs(H) + np.abs(Q) * (1.1 * aG * np.abs(U) + np.abs(G * sg) * aU
                                                        + np.abs(H))).sum(1),
                      wg=np.abs(dG).T @ np.abs(x), wu=np.abs(dU).T @ np.abs(x),
                      wd=np.abs(dy).T @ np.abs(s * H))
    return out


def layer_backward(x, dy, Z, ids, wr, wg, wu, wd, shared=None, grad=None):
    """Gradients of the layer for given logits and selection.  Returns (out, mag)
    with keys x, logits, w_router, w_gate, w_up, w_down, ws_gate, ws_up, ws_down
    as far as they exist.  ids outside [0, E) contribute nothing."""
    N, d = x.shape
    E = Z.shape[1]
    x64 = x.astype(np.float64)
    out = dict(x=np.zeros((N, d)), logits=np.zeros((N, E)) if grad is None else grad.astype(np.float64),
               w_gate=np.zeros(wg.shape), w_up=np.zeros(wu.shape), w_down=np.zeros(wd.shape))
    mag = {k: np.zeros(v.shape) for k, v in out.items()}
    t_of, k_of = np.nonzero((ids >= 0) & (ids < E))
    e_of = ids[t_of, k_of]
    for e in range(E):
        t = t_of[e_of == e]
        if t.size == 0:
            continue
        s = _sigmoid(Z[t, e].astype(np.float64))
        r = expert_backward(x[t], dy[t], s, wg[e], wu[e], wd[e])
        slope = s * _sigmoid(-Z[t, e].astype(np.float64))
        for o, q in ((out, r), (mag, r["mag"])):
            np.add.at(o["x"], t, q["dx"])
            np.add.at(o["logits"], (t, np.full(t.size, e)), q["ds"] * slope)
            o["w_gate"][e], o["w_up"][e], o["w_down"][e] = q["wg"], q["wu"], q["wd"]
    if shared is not None:
        r = expert_backward(x, dy, np.ones(N), *shared)
        for o, q in ((out, r), (mag, r["mag"])):
            o["x"] += q["dx"]
            o["ws_gate"], o["ws_up"], o["ws_down"] = (q[k][None] for k in ("wg", "wu", "wd"))
    if wr is not None:
        w64 = wr.astype(np.float64)
        out["x"] += out["logits"] @ w64
        out["w_router"] = out["logits"].T @ x64
        mag["x"] += np.abs(out["logits"]) @ np.abs(w64)
        mag["w_router"] = np.abs(out["logits"]).T @ np.abs(x64)
    return out, mag

"""Cases of the operators around the MoE layer: the root-mean-square norm of the
residual stream (with its addition, the sandwich form and an E4M3 output), the
balance loss of the router, both with their gradients, and the gradients of
the layer itself.

``run`` computes a case in its plain form (elementary torch operations in
32 bits), or with ``own`` set through the package's entry points.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
COEF = 1e-2


# ---------------------------------------------------------------- the cases
def norm_case(name, direction, rows, d, residual, post, quant, weight):
    """direction: fwd or bwd; residual: none, bf16 or f32 (the type of the
    residual stream); post: a second norm on x before the addition; quant: the
    output also as E4M3 codes with one scale per 1 x 128 group; weight: type of
    the weights."""
    case = {"op": "norm", "direction": direction, "rows": rows, "d": d, "residual": residual,
            "post": post, "quant": quant, "weight": weight}
    return dict(case, name=name) if name else case


def balance_case(name, direction, N, E, K, score, segments, add):
    """direction: fwd, or step (loss and gradient); segments: sequences in the
    batch (0: the whole batch is one, without gaps); add: the gradient is added
    to one that is there already."""
    case = {"op": "balance", "direction": direction, "N": N, "E": E, "K": K, "score": score,
            "segments": segments, "add": add}
    return dict(case, name=name) if name else case


def layer_case(name, N, d, E, K, h, shared, add):
    """Backward pass of the layer: shared: hidden width of the shared expert (0:
    none); add: the logits have a gradient of their own already (a balance loss)."""
    case = {"op": "layer", "N": N, "d": d, "E": E, "K": K, "h": h, "shared": shared, "add": add}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one sequence being decoded: the norm in front of an E4M3 layer, latency alone
        norm_case("norm token", "fwd", 1, 2560, "bf16", False, True, "bf16"),
        # a decode batch, 64 tokens, between two sandwich-normed sublayers
        norm_case("norm decode", "fwd", 64, 2560, "f32", True, True, "bf16"),
        # an odd width that no vector load fits, a ragged row count, no residual
        norm_case("norm odd", "fwd", 3001, 777, "none", False, False, "f32"),
        # the largest batch in front of the E4M3 layer, fp32 residual stream
        norm_case("norm large", "fwd", 65536, 2560, "f32", True, True, "f32"),
        # odd width, sandwich form, all four gradients
        norm_case("norm grad odd", "bwd", 1025, 1001, "bf16", True, False, "f32"),
        # a training microbatch of the wide layer, fp32 residual stream, sandwich form
        norm_case("norm grad large", "bwd", 16384, 2560, "f32", True, False, "f32"),
        # a small batch of the narrow layer, one segment, for logging: latency
        balance_case("balance small", "fwd", 256, 128, 8, "sigmoid", 0, False),
        # odd sizes, softmax scores, short and empty sequences, padding between them
        balance_case("balance odd step", "step", 1237, 100, 5, "softmax", 9, False),
        # the largest training batch, gradient added to the router's own
        balance_case("balance step", "step", 65536, 384, 6, "sigmoid_norm", 16, True),
        # a short microbatch, odd token count, of a small layer without a shared expert
        layer_case("layer grad small", 333, 320, 20, 4, 160, 0, False),
        # a microbatch of the narrower layer
        layer_case("layer grad narrow", 4096, 2048, 128, 8, 768, 768, False),
        # a training microbatch of the wide layer, balance loss on
        layer_case("layer grad wide", 16384, 2560, 384, 6, 512, 512, True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw_norm(rng):
    direction = rng.choice(["fwd", "fwd", "bwd"])
    quant = direction == "fwd" and rng.random() < 0.6
    d = 128 * log_int(rng, 1, 64) if quant else log_int(rng, 64, 8192)
    most = 65536 * 2560 if direction == "fwd" else 16384 * 2560
    rows = log_int(rng, 1, min(65536, most // d))
    return norm_case(None, direction, rows, d, rng.choice(["none", "bf16", "f32"]),
                     rng.random() < 0.5, quant, rng.choice(["bf16", "f32"]))


def draw_balance(rng):
    return balance_case(None, rng.choice(["fwd", "step"]), log_int(rng, 1, 65536),
                        log_int(rng, 9, 384), rng.randint(1, 8),
                        rng.choice(["sigmoid", "sigmoid_norm", "softmax"]),
                        rng.choice([0, log_int(rng, 1, 64)]), rng.random() < 0.5)


def draw_layer(rng):
    d, h, E = 64 * log_int(rng, 1, 40), 32 * log_int(rng, 1, 24), log_int(rng, 9, 384)
    if d * h * E > 2560 * 512 * 384:
        h = 32
    K = rng.randint(1, 8)
    most = 16384 * 6 * 2560 * 512 // (K * d * h)
    return layer_case(None, log_int(rng, 1, min(16384, most)), d, E, K, h,
                      rng.choice([0, h, 32 * log_int(rng, 1, 16)]), rng.random() < 0.5)


def draw(rng):
    return rng.choice([draw_norm, draw_balance, draw_layer])(rng)


# ---------------------------------------------------------------- inputs
def stream_dtype(case):
    return torch.float32 if case["residual"] == "f32" else torch.bfloat16


def prepare_norm(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    rows, d = case["rows"], case["d"]
    wt = torch.bfloat16 if case["weight"] == "bf16" else torch.float32
    # a residual stream has a few channels far above the others
    channel = 1.0 + 30.0 * (torch.rand(d, generator=g, device="cuda") < 0.004)
    s = {"case": case, "x": (0.7 * rand(rows, d)).bfloat16(),
         "weight": (1.0 + 0.2 * rand(d)).to(wt),
         "post_weight": (0.5 + 0.1 * rand(d)).to(wt) if case["post"] else None, "residual": None}
    if case["residual"] != "none":
        s["residual"] = (2.0 * rand(rows, d) * channel).to(stream_dtype(case))
    if case["direction"] == "bwd":
        s["dy"] = (1e-2 * rand(rows, d)).bfloat16()
        if case["residual"] != "none":
            # what the forward pass left, and the gradient from the layers above
            s["r"] = (s.pop("residual").float() + s["x"].float()).to(stream_dtype(case))
            s["dres"] = (1e-2 * rand(rows, d)).to(stream_dtype(case))
        elif case["post"]:
            s["r"] = (0.5 * rand(rows, d) * channel).bfloat16()
            s["dres"] = None
        else:
            s["r"], s["dres"] = s["x"], None
    return s


def prepare_balance(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, E, K = case["N"], case["E"], case["K"]
    popular = 0.8 * torch.randn(E, generator=g, device="cuda")
    logits = 1.5 * torch.randn(N, E, generator=g, device="cuda") + popular
    beta = 0.1 * torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(logits + beta, K, dim=1).indices.int()
    s = {"case": case, "logits": logits, "ids": ids, "begin": None, "end": None, "grad": None,
         "grad_loss": None}
    G = case["segments"]
    if G:
        # cut points of G sequences with a little padding behind each; some are empty
        cut = torch.rand(G - 1, generator=g, device="cuda").mul(N + 1).long().sort().values
        edge = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), N)])
        begin, room = edge[:-1], edge[1:] - edge[:-1]
        pad = torch.rand(G, generator=g, device="cuda").mul(0.1 * room).long()
        s["begin"], s["end"] = begin.int(), (begin + room - pad).int()
    if case["direction"] == "step":
        s["grad_loss"] = torch.full((1,), 0.5, device="cuda")
        if case["add"]:
            s["grad"] = 1e-7 * torch.randn(N, E, generator=g, device="cuda")
    return s


def prepare_layer(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(std, *shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)

    N, d, E, K, h, hs = (case[k] for k in ("N", "d", "E", "K", "h", "shared"))
    s = {"case": case, "x": rand(1.0, N, d), "dy": rand(1e-3, N, d),
         "w_router": rand(1.5 / math.sqrt(d), E, d), "w_gate": rand(1.0 / math.sqrt(d), E, h, d),
         "w_up": rand(1.0 / math.sqrt(d), E, h, d), "w_down": rand(1.0 / math.sqrt(h), E, d, h)}
    s["ws_gate"] = rand(1.0 / math.sqrt(d), 1, hs, d) if hs else None
    s["ws_up"] = rand(1.0 / math.sqrt(d), 1, hs, d) if hs else None
    s["ws_down"] = rand(1.0 / math.sqrt(hs), 1, d, hs) if hs else None
    # what the forward pass left: logits, and the experts that a bias chose which
    # keeps the loads near each other, as the quantile update does
    popular = 0.8 * torch.randn(E, generator=g, device="cuda")
    s["logits"] = s["x"].float() @ s["w_router"].float().t() + popular
    off = 0.15 * torch.randn(E, generator=g, device="cuda")
    s["ids"] = torch.topk(s["logits"] - popular + off, K, dim=1).indices.int()
    s["grad"] = 1e-3 * torch.randn(N, E, generator=g, device="cuda") if case["add"] else None
    return s


PREPARE = {"norm": prepare_norm, "balance": prepare_balance, "layer": prepare_layer}


def prepare(case, seed):
    return PREPARE[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def plain_norm(s):
    case = s["case"]
    u = s["x"].float()
    if case["post"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * s["post_weight"].float()
    r = u if s["residual"] is None else u + s["residual"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {"y": y.bfloat16()}
    if case["residual"] != "none" or case["post"]:
        out["r"] = r.to(stream_dtype(case))
    if case["quant"]:
        group = y.view(y.shape[0], -1, 128)
        scale = group.abs().amax(-1, keepdim=True) / 448.0
        code = torch.where(scale > 0, group / scale, torch.zeros_like(group)).clamp(-448.0, 448.0)
        out["codes"] = code.to(torch.float8_e4m3fn).view(y.shape)
        out["scales"] = scale.squeeze(-1)
    return out


def plain_norm_grad(s):
    r, dy, w = s["r"].float(), s["dy"].float(), s["weight"].float()
    a = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    n, h = r * a, dy * w
    dr = a * (h - n * (h * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dr = dr + s["dres"].float()
    out = {"dweight": (dy * n).sum(0)}
    if s["case"]["post"]:
        x = s["x"].float()
        b = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        m, k = x * b, dr * s["post_weight"].float()
        out["dx"] = (b * (k - m * (k * m).mean(-1, keepdim=True))).bfloat16()
        out["dpost"] = (dr * m).sum(0)
    else:
        out["dx"] = dr.bfloat16()
    if s["case"]["residual"] != "none":
        out["dresidual"] = dr.to(stream_dtype(s["case"]))
    return out


def segment_of(s):
    """The segment of every row, and 1 or 0 for rows inside and outside of one."""
    N = s["logits"].shape[0]
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    if s["begin"] is None:
        return torch.zeros_like(t).long(), torch.ones(N, device="cuda")
    g = torch.searchsorted(s["begin"], t, right=True) - 1
    inside = (g >= 0) & (t < s["end"][g.clamp(min=0)])
    return g.clamp(min=0), inside.float()


def plain_balance(s):
    case, z = s["case"], s["logits"]
    G, E, K = max(case["segments"], 1), case["E"], case["K"]
    g, inside = segment_of(s)
    live = inside.unsqueeze(1)
    if case["score"] == "softmax":
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        sig = 1.0 / (1.0 + torch.exp(-z))
        den = sig.sum(-1, keepdim=True) if case["score"] == "sigmoid_norm" else 1.0
        p = sig / den
    member = (g.unsqueeze(0) == torch.arange(G, device="cuda").unsqueeze(1)).float() * inside
    length = member.sum(1, keepdim=True)
    mean = (member @ p) / length.clamp(min=1.0)
    flat = (g.unsqueeze(1) * E + s["ids"]).reshape(-1)
    counts = torch.zeros(G * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, flat, live.int().expand(-1, K).reshape(-1))
    counts = counts.view(G, E)
    f = counts.float() * (E / counts.sum(1, keepdim=True).clamp(min=1).float())
    out = {"loss": COEF / G * (f * mean).sum().reshape(1), "counts": counts, "mean": mean}
    if case["direction"] == "step":
        ft = f[g]
        scale = live * (COEF / G) * s["grad_loss"] / length[g].clamp(min=1.0)
        if case["score"] == "sigmoid":
            dz = scale * ft * p * (1.0 - p)
        else:
            slope = p if case["score"] == "softmax" else p * (1.0 - sig)
            dz = scale * slope * (ft - (ft * p).sum(-1, keepdim=True))
        out["dlogits"] = dz if s["grad"] is None else dz + s["grad"]
    return out


def plain_experts_grad(x, dy, scale, w_gate, w_up, w_down):
    """Gradients of scale * (silu(x Wg^T) * (x Wu^T)) Wd^T for every expert's rows
    [E, rows, d]: of x, of the scale and of the three weights."""
    wg, wu, wd = w_gate.float(), w_up.float(), w_down.float()
    gate, up = torch.bmm(x, wg.mT.contiguous()), torch.bmm(x, wu.mT.contiguous())
    sig = 1.0 / (1.0 + torch.exp(-gate))
    hidden = gate * sig * up
    back = torch.bmm(dy, wd)
    dscale = (back * hidden).sum(-1)
    back = back * scale.unsqueeze(-1)
    dup = back * gate * sig
    dgate = back * up * sig * (1.0 + gate * (1.0 - sig))
    dx = torch.bmm(dgate, wg) + torch.bmm(dup, wu)
    grads = [torch.bmm(dgate.mT.contiguous(), x), torch.bmm(dup.mT.contiguous(), x),
             torch.bmm(dy.mT.contiguous(), hidden * scale.unsqueeze(-1))]
    return dx, dscale, [t.bfloat16() for t in grads]


def plain_layer_grad(s):
    case = s["case"]
    N, d, E, K = case["N"], case["d"], case["E"], case["K"]
    x, dy = s["x"].float(), s["dy"].float()
    ids = s["ids"].long()
    z = torch.gather(s["logits"], 1, ids)
    score = 1.0 / (1.0 + torch.exp(-z))
    # the pairs of every expert side by side, padded to the longest expert's
    flat = ids.reshape(-1)
    loads = torch.bincount(flat, minlength=E)
    most = int(loads.max())
    order = torch.argsort(flat, stable=True)
    rank = torch.arange(N * K, device="cuda") - (loads.cumsum(0) - loads)[flat[order]]
    slot = torch.empty_like(order)
    slot[order] = flat[order] * most + rank
    token = torch.arange(N, device="cuda").repeat_interleave(K)
    xp, dyp = x.new_zeros(E * most, d), x.new_zeros(E * most, d)
    sp = x.new_zeros(E * most)
    xp[slot], dyp[slot], sp[slot] = x[token], dy[token], score.reshape(-1)
    dxp, dscore, grads = plain_experts_grad(xp.view(E, most, d), dyp.view(E, most, d),
                                            sp.view(E, most), s["w_gate"], s["w_up"], s["w_down"])
    dx = dxp.view(E * most, d)[slot].view(N, K, d).sum(1)
    dscore = dscore.view(-1)[slot].view(N, K)
    dz = torch.zeros_like(s["logits"]) if s["grad"] is None else s["grad"].clone()
    dz.scatter_add_(1, ids, dscore * score * (1.0 / (1.0 + torch.exp(z))))
    out = dict(zip(("w_gate", "w_up", "w_down"), grads))
    if case["shared"]:
        one = torch.ones(1, N, device="cuda")
        dxs, _, grads = plain_experts_grad(x.unsqueeze(0), dy.unsqueeze(0), one, s["ws_gate"],
                                           s["ws_up"], s["ws_down"])
        dx = dx + dxs[0]
        out.update(zip(("ws_gate", "ws_up", "ws_down"), grads))
    out["dx"] = (dx + dz @ s["w_router"].float()).bfloat16()
    out["w_router"] = (dz.t() @ x).bfloat16()
    out["dlogits"] = dz
    return out


# ---------------------------------------------------------------- the package's operators
def own_norm(s):
    import sigmoid_top_routing_router_amd as M
    case = s["case"]
    y, r, q = M.rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"],
                         post_weight=s["post_weight"], quantize=case["quant"])
    out = {"y": y}
    if r is not None:
        out["r"] = r
    if q is not None:
        out["codes"], out["scales"] = q[0].view(torch.float8_e4m3fn), q[1]
    return out


def own_norm_grad(s):
    import sigmoid_top_routing_router_amd as M
    dx, dres, dw, dpost = M.rms_norm_backward(
        s["dy"], s["r"], s["weight"], eps=EPS, grad_residual=s["dres"],
        x=s["x"] if s["case"]["post"] else None, post_weight=s["post_weight"])
    out = {"dx": dx, "dweight": dw}
    if s["case"]["post"]:
        out["dpost"] = dpost
    if s["case"]["residual"] != "none":
        out["dresidual"] = dres
    return out


def own_balance(s):
    import sigmoid_top_routing_router_amd as M
    case = s["case"]
    segments = None if s["begin"] is None else (s["begin"], s["end"])
    loss, counts, mean = M.balance_loss(s["logits"], s["ids"], coef=COEF, score=case["score"],
                                        segments=segments)
    out = {"loss": loss, "counts": counts, "mean": mean}
    if case["direction"] == "step":
        out["dlogits"] = M.balance_loss_backward(s["logits"], counts, coef=COEF,
                                                 score=case["score"], segments=segments,
                                                 grad_loss=s["grad_loss"], grad_logits=s["grad"])
    return out


def own_layer_grad(s):
    import sigmoid_top_routing_router_amd as M
    names = ["w_router", "w_gate", "w_up", "w_down"]
    names += ["ws_gate", "ws_up", "ws_down"] if s["case"]["shared"] else []
    dx, dlogits, grads = M.backward(s["dy"], s["x"], M.ExpertWeights(**{n: s[n] for n in names}),
                                    s["logits"], s["ids"], grad_logits=s["grad"])
    return {"dx": dx, "dlogits": dlogits, **{n: getattr(grads, n) for n in names}}


def run(state):
    case = state["case"]
    if case["op"] == "balance":
        return own_balance(state) if own else plain_balance(state)
    if case["op"] == "layer":
        return own_layer_grad(state) if own else plain_layer_grad(state)
    if case["direction"] == "bwd":
        return own_norm_grad(state) if own else plain_norm_grad(state)
    return own_norm(state) if own else plain_norm(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n, d = case["rows"] * case["d"], case["d"]
        stream = 0 if case["residual"] == "none" else 4 if case["residual"] == "f32" else 2
        weights = (2 if case["post"] else 1) * d * (4 if case["weight"] == "f32" else 2)
        if case["direction"] == "fwd":
            kept = stream or (2 if case["post"] else 0)  # the sum that leaves
            moved = n * (2 + stream + kept + 2) + weights
            if case["quant"]:
                moved += n + n // 128 * 4
            return {"bytes": moved, "flops": n * (12 if case["post"] else 8)}
        # dy, r, dx; the gradient from above and the one passed on; x of the sandwich form
        moved = n * (2 + (stream or 2) + 2 + 2 * stream + (2 if case["post"] else 0))
        moved += weights + (2 if case["post"] else 1) * d * 4
        return {"bytes": moved, "flops": n * (28 if case["post"] else 14)}
    if case["op"] == "layer":
        N, d, E, K, h, hs = (case[k] for k in ("N", "d", "E", "K", "h", "shared"))
        # x, dy and dx; the weights of the experts that are used, and every weight's gradient;
        # the hidden products of the forward pass are formed again: eight products of each pair
        used = E * (1.0 - (1.0 - K / E) ** N)
        moved = 3 * N * d * 2 + N * E * 4 * (2 if case["add"] else 1) + 2 * N * K * 4 + 4 * E * d
        moved += 6 * d * h * (used + E) + 12 * d * hs
        flops = 16 * d * (N * K * h + N * hs) + 4 * N * E * d
        return {"bytes": moved, "flops": flops}
    N, E, K, G = case["N"], case["E"], case["K"], max(case["segments"], 1)
    moved = N * E * 4 + N * K * 4 + G * E * 8 + G * 8
    flops = N * E * 6
    if case["direction"] == "step":
        # the gradient needs the loads of the whole segment: the logits once more
        moved += N * E * 4 * (2 + (1 if case["add"] else 0))
        flops += N * E * 12
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- from the definitions, 64 bits
def unit_rms(v):
    """v over its root mean square, and that root's reciprocal, row by row."""
    inv = 1.0 / torch.sqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / v.shape[-1] + EPS)
    return v * inv, inv


def norm_pullback(v, grad):
    """The gradient of v through v / rms(v)."""
    unit, inv = unit_rms(v)
    along = torch.einsum("td,td->t", unit, grad).unsqueeze(1) / v.shape[-1]
    return inv * (grad - along * unit)


def exact_norm(s, case):
    x, w = s["x"].double(), s["weight"].double()
    if case["direction"] == "fwd":
        total = unit_rms(x)[0] * s["post_weight"].double() if case["post"] else x
        if s["residual"] is not None:
            total = s["residual"].double() + total
        y = unit_rms(total)[0] * w
        out = {"y": y}
        if case["residual"] != "none" or case["post"]:
            out["r"] = total
        if case["quant"]:
            blocks = y.unflatten(1, (-1, 128))
            top = torch.maximum(blocks.amax(2), -blocks.amin(2)) / 448
            out["scales"] = top
            out["codes"] = (blocks / top.unsqueeze(2)).flatten(1)  # before the rounding to E4M3
        return out
    r, dy = s["r"].double(), s["dy"].double()
    through = norm_pullback(r, dy * w)
    if s["dres"] is not None:
        through = s["dres"].double() + through
    out = {"dweight": torch.einsum("td,td->d", dy, unit_rms(r)[0])}
    out["dx"] = through
    if case["post"]:
        out["dx"] = norm_pullback(x, through * s["post_weight"].double())
        out["dpost"] = torch.einsum("td,td->d", through, unit_rms(x)[0])
    if case["residual"] != "none":
        out["dresidual"] = through
    return out


def exact_balance(s, case):
    N, E, G = case["N"], case["E"], max(case["segments"], 1)
    spans = [(0, N)] if s["begin"] is None else list(zip(s["begin"].tolist(), s["end"].tolist()))
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    counts, mean = [], []
    grad = torch.zeros(N, E, dtype=torch.float64, device="cuda") if s["grad"] is None else s["grad"].double()
    for lo, hi in spans:
        c = torch.bincount(s["ids"][lo:hi].reshape(-1), minlength=E)
        counts.append(c.int())
        if hi <= lo:
            mean.append(torch.zeros(E, dtype=torch.float64, device="cuda"))
            continue
        z = s["logits"][lo:hi].double().requires_grad_(True)
        score = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
        if case["score"] == "sigmoid_norm":
            score = score / score.sum(1, keepdim=True)
        average = score.mean(0)
        part = COEF / G * E * torch.dot(c.double() / c.sum(), average)
        if case["direction"] == "step":
            grad[lo:hi] += s["grad_loss"].double() * torch.autograd.grad(part, z)[0]
        loss = loss + part.detach()
        mean.append(average.detach())
    out = {"loss": loss, "counts": torch.stack(counts), "mean": torch.stack(mean)}
    if case["direction"] == "step":
        out["dlogits"] = grad
    return out


def swiglu(x, w_gate, w_up, w_down):
    return (torch.nn.functional.silu(x @ w_gate.t()) * (x @ w_up.t())) @ w_down.t()


def exact_layer(s, case):
    """Automatic differentiation of <dy, y>, expert by expert."""
    x, dy = s["x"].double(), s["dy"].double()
    dx = torch.zeros_like(x)
    dlogits = torch.zeros_like(s["logits"], dtype=torch.float64) if s["grad"] is None else s["grad"].double()
    out = {n: torch.zeros(s[n].shape, dtype=torch.float32, device="cuda") for n in ("w_gate", "w_up", "w_down")}

    def pull(rows, z, weights):
        """Adds this expert's part to dx; its weights' gradients and the logits'."""
        xe = x[rows].requires_grad_(True)
        ws = [w.double().requires_grad_(True) for w in weights]
        score = torch.sigmoid(z).unsqueeze(1) if z is not None else 1.0
        y = torch.sum(dy[rows] * score * swiglu(xe, *ws))
        grads = torch.autograd.grad(y, [xe, *ws] + ([z] if z is not None else []))
        dx.index_add_(0, rows, grads[0])
        return grads[1:4], grads[4] if z is not None else None

    for e in range(case["E"]):
        rows = (s["ids"] == e).any(1).nonzero().squeeze(1)
        if rows.numel():
            z = s["logits"][rows, e].double().requires_grad_(True)
            grads, dz = pull(rows, z, (s["w_gate"][e], s["w_up"][e], s["w_down"][e]))
            dlogits[rows, e] += dz
            for n, g in zip(("w_gate", "w_up", "w_down"), grads):
                out[n][e] = g
    if case["shared"]:
        grads, _ = pull(torch.arange(case["N"], device="cuda"), None,
                        (s["ws_gate"][0], s["ws_up"][0], s["ws_down"][0]))
        for n, g in zip(("ws_gate", "ws_up", "ws_down"), grads):
            out[n] = g.unsqueeze(0)
    out["dx"] = dx + dlogits @ s["w_router"].double()
    out["w_router"] = dlogits.t() @ x
    out["dlogits"] = dlogits
    return out


EXACT = {"norm": exact_norm, "balance": exact_balance, "layer": exact_layer}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed), case)

"""Cases of the operators with which a caller takes the MoE layer apart: tokens
sorted by expert and back again (with the mixture weights and the shared
expert's output applied), the gradients of both, the same with activations
that are kept in 8 bits for the backward pass, and the experts' products in
8-bit integers with a scale for each token and each output channel.

``run`` computes a case in its plain form (elementary torch operations in
32 bits), or with ``own`` set through the package's entry points.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
GROUP = 128  # values of a row that share a scale in E4M3


# ---------------------------------------------------------------- the cases
def sort_case(name, direction, N, d, E, K, rows, away):
    """direction: fwd (grouping and sorted rows), or bwd (gradient of the
    tokens); rows: type of the tokens, bf16, f32 or e4m3 (kept in 8 bits, the
    sorted rows are bf16); away: half of the experts are on other GPUs, their
    pairs have ids outside of [0, E)."""
    case = {"op": "sort", "direction": direction, "N": N, "d": d, "E": E, "K": K, "rows": rows,
            "away": away}
    return dict(case, name=name) if name else case


def back_case(name, direction, N, d, E, K, rows, weights, base, kept, away):
    """rows: type of the expert rows, bf16 or f32; weights: mixture weights are
    applied; base: the shared expert's output is added; kept: forward also
    leaves the rows as E4M3 codes, backward reads those in their place."""
    case = {"op": "back", "direction": direction, "N": N, "d": d, "E": E, "K": K, "rows": rows,
            "weights": weights, "base": base, "kept": kept, "away": away}
    return dict(case, name=name) if name else case


def int8_case(name, N, k, cols, E, K, swiglu, gather):
    """N tokens, k deep, cols output columns.  E: experts, K of them a token (E
    0: one dense product); swiglu: silu(x Wg^T) * (x Wu^T) of two weights;
    gather: the product picks its rows from the tokens (else it is given sorted
    rows)."""
    case = {"op": "int8", "N": N, "k": k, "cols": cols, "E": E, "K": K, "swiglu": swiglu,
            "gather": gather}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one sequence being decoded, its token to the experts: latency alone
        sort_case("sort token", "fwd", 1, 2560, 384, 6, "bf16", False),
        # fp32 rows of an odd width, half of the experts on other GPUs
        sort_case("sort odd", "fwd", 1237, 777, 100, 5, "f32", True),
        # a training microbatch of the wide layer on its way to the experts
        sort_case("sort large", "fwd", 16384, 2560, 384, 6, "bf16", False),
        # the same rows once more in the backward pass, from tokens kept in 8 bits
        sort_case("sort kept", "fwd", 16384, 2560, 384, 6, "e4m3", False),
        # gradient of that microbatch's tokens
        sort_case("sort grad", "bwd", 16384, 2560, 384, 6, "bf16", False),
        # a decode batch, 64 tokens, on its way back
        back_case("back decode", "fwd", 64, 2560, 384, 6, "bf16", True, True, False, False),
        # the microbatch on its way back, its expert rows kept in 8 bits
        back_case("back kept", "fwd", 16384, 2560, 384, 6, "bf16", True, True, True, False),
        # gradients of fp32 rows of an odd width, half of the experts elsewhere
        back_case("back grad odd", "bwd", 1237, 777, 100, 5, "f32", True, False, False, True),
        # gradients of the microbatch's expert rows and weights, from the kept rows
        back_case("back grad kept", "bwd", 16384, 2560, 384, 6, "bf16", True, False, True, False),
        # one token through its experts' gate and up products: weights read once
        int8_case("int8 token", 1, 2560, 512, 384, 6, True, True),
        # a prefill batch through the experts' gate and up products
        int8_case("int8 experts", 16384, 2560, 512, 384, 6, True, True),
        # one dense product of a long prefill
        int8_case("int8 dense", 8192, 8192, 8192, 0, 1, False, False),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw_rows(rng):
    """Tokens, width, experts, experts a token, type of the rows, kept in 8 bits."""
    kept = rng.random() < 0.4
    d = 128 * log_int(rng, 1, 64) if kept else log_int(rng, 64, 8192)
    K = rng.randint(1, 8)
    rows = "bf16" if kept else rng.choice(["bf16", "f32"])
    most = 16384 * 6 * 2560 // (K * d * (2 if rows == "f32" else 1))
    return log_int(rng, 1, min(65536, most)), d, log_int(rng, 9, 384), K, rows, kept


def draw_sort(rng):
    N, d, E, K, rows, kept = draw_rows(rng)
    direction = "fwd" if kept else rng.choice(["fwd", "bwd"])
    return sort_case(None, direction, N, d, E, K, "e4m3" if kept else rows, rng.random() < 0.3)


def draw_back(rng):
    N, d, E, K, rows, kept = draw_rows(rng)
    direction = rng.choice(["fwd", "bwd"])
    return back_case(None, direction, N, d, E, K, rows, direction == "bwd" or rng.random() < 0.8,
                     direction == "fwd" and rng.random() < 0.5, kept,
                     not kept and rng.random() < 0.3)


def draw_int8(rng):
    if rng.random() < 0.4:
        N, k, cols = log_int(rng, 1, 16384), 16 * log_int(rng, 4, 512), 8 * log_int(rng, 4, 1024)
        N = max(1, min(N, 8192 ** 3 // (2 * k * cols)))
        return int8_case(None, N, k, cols, 0, 1, rng.random() < 0.5, False)
    K, E = rng.randint(1, 8), log_int(rng, 9, 384)
    k, cols = 16 * log_int(rng, 4, 160), 8 * log_int(rng, 4, 96)
    if k * cols * E > 2560 * 512 * 384:
        cols = 32
    N = log_int(rng, 1, min(16384, 16384 * 6 * 2560 * 512 // (K * k * cols)))
    return int8_case(None, N, k, cols, E, K, rng.random() < 0.5, rng.random() < 0.5)


def draw(rng):
    return rng.choice([draw_sort, draw_back, draw_int8])(rng)


# ---------------------------------------------------------------- inputs
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.bfloat16}


def choose(g, N, E, K, away=False):
    """K experts for every token: popular ones and a bias that nearly levels the
    loads, as the quantile update does; away: E of 2 E experts are here."""
    every = 2 * E if away else E
    popular = 0.25 * torch.randn(every, generator=g, device="cuda")
    score = torch.randn(N, every, generator=g, device="cuda") + popular
    ids = torch.topk(score, K, dim=1).indices.int()
    return ids - E // 2 if away else ids


def group(ids, E):
    """Counts, offsets, the pairs in sorted order and every pair's place there
    (-1 behind the last sorted pair and for pairs whose expert is elsewhere)."""
    flat = ids.reshape(-1).long()
    here = (flat >= 0) & (flat < E)
    key = torch.where(here, flat, E)
    order = torch.argsort(key, stable=True)
    counts = (key.unsqueeze(0) == torch.arange(E, device="cuda").unsqueeze(1)).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(flat.numel(), device="cuda")
    pos = torch.empty_like(order)
    pos[order] = place
    return {"counts": counts.int(), "offsets": offsets.int(),
            "sorted_src": torch.where(place < offsets[-1], order, -1).int(),
            "src_pos": torch.where(here, pos, -1).int().view(ids.shape)}


def e4m3(x):
    """E4M3 codes and one fp32 scale for each group of a row."""
    parts = x.float().unflatten(1, (-1, GROUP))
    scale = parts.abs().amax(-1, keepdim=True) / E4M3_MAX
    code = torch.where(scale > 0, parts / scale, torch.zeros_like(parts))
    code = code.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return code.view(x.shape), scale.squeeze(-1)


def prepare_rows(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, d, E, K = (case[k] for k in ("N", "d", "E", "K"))
    t = TYPES[case["rows"]]

    def rand(std, *shape):
        return torch.empty(*shape, dtype=t, device="cuda").normal_(0.0, std, generator=g)

    # activations have a few channels far above the others
    channel = (1.0 + 30.0 * (torch.rand(d, generator=g, device="cuda") < 0.004)).to(t)
    s = {"case": case, "ids": choose(g, N, E, K, case["away"])}
    s.update(group(s["ids"], E))
    if case["op"] == "sort":
        if case["direction"] == "bwd":
            s["grad_rows"] = rand(1e-2, N * K, d)
            return s
        s["x"] = rand(1.0, N, d) * channel
        if case["rows"] == "e4m3":
            s["x"] = e4m3(s["x"])
        # with experts elsewhere the sorted rows are fewer than the buffer's
        s["out"] = torch.zeros(N * K, d, dtype=t, device="cuda") if case["away"] else None
        return s
    score = torch.randn(N, K, generator=g, device="cuda")
    s["weights"] = 1.0 / (1.0 + torch.exp(-score)) if case["weights"] else None
    rows = rand(0.5, N * K, d) * channel
    if case["direction"] == "fwd":
        s["expert_rows"] = rows
        s["base"] = rand(0.5, N, d) if case["base"] else None
        return s
    s["grad_y"] = rand(1e-2, N, d)
    s["expert_rows"] = e4m3(rows) if case["kept"] else rows
    s["out"] = torch.zeros(N * K, d, dtype=t, device="cuda") if case["away"] else None
    return s


def prepare_int8(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, k, cols, E, K = (case[n] for n in ("N", "k", "cols", "E", "K"))

    def weight():
        """Codes of normal weights whose largest in a channel is about four times
        their spread, and the channels' scales."""
        codes = torch.empty(max(E, 1), cols, k, dtype=torch.int8, device="cuda")
        for e in range(max(E, 1)):
            v = torch.randn(cols, k, generator=g, device="cuda")
            codes[e] = (v * 31.75).round_().clamp_(-127.0, 127.0)
        scale = torch.rand(max(E, 1), cols, generator=g, device="cuda") * 0.4 + 0.8
        scale = scale / (31.75 * math.sqrt(k))
        return (codes, scale) if E else (codes[0], scale[0])

    s = {"case": case, "w": weight(), "w_up": weight() if case["swiglu"] else None}
    rows = N if case["gather"] or not E else N * K
    channel = (1.0 + 30.0 * (torch.rand(k, generator=g, device="cuda") < 0.004)).bfloat16()
    s["x"] = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.0, generator=g) * channel
    if E:
        s["ids"] = choose(g, N, E, K)
        s.update(group(s["ids"], E))
    return s


def prepare(case, seed):
    return prepare_int8(case, seed) if case["op"] == "int8" else prepare_rows(case, seed)


# ---------------------------------------------------------------- plain forms
def kept_values(pair):
    """What E4M3 codes and their scales stand for, in fp32."""
    codes, scales = pair
    return (codes.float().unflatten(1, (-1, GROUP)) * scales.unsqueeze(-1)).flatten(1)


def plain_sort(s):
    case = s["case"]
    if case["direction"] == "bwd":
        pos = s["src_pos"].long()
        parts = s["grad_rows"].float()[pos.clamp(min=0)]
        parts = torch.where((pos >= 0).unsqueeze(-1), parts, torch.zeros_like(parts))
        return {"grad_x": parts.sum(1).to(s["grad_rows"].dtype)}
    out = group(s["ids"], case["E"])
    src = out["sorted_src"].long()
    x = kept_values(s["x"]).bfloat16() if case["rows"] == "e4m3" else s["x"]
    rows = x[src.clamp(min=0) // case["K"]]
    if s["out"] is not None:
        rows = torch.where((src >= 0).unsqueeze(1), rows, s["out"])
    out["rows"] = rows
    return out


def plain_back(s):
    case = s["case"]
    pos, t = s["src_pos"].long(), TYPES[case["rows"]]
    here = (pos >= 0).unsqueeze(-1)
    if case["direction"] == "fwd":
        parts = s["expert_rows"].float()[pos.clamp(min=0)]
        if s["weights"] is not None:
            parts = parts * s["weights"].unsqueeze(-1)
        y = torch.where(here, parts, torch.zeros_like(parts)).sum(1)
        if s["base"] is not None:
            y = y + s["base"].float()
        out = {"y": y.to(t)}
        if case["kept"]:
            out["codes"], out["scales"] = e4m3(s["expert_rows"])
        return out
    rows = kept_values(s["expert_rows"]) if case["kept"] else s["expert_rows"].float()
    dy = s["grad_y"].float()
    dots = (rows[pos.clamp(min=0)] * dy.unsqueeze(1)).sum(-1)
    src = s["sorted_src"].long()
    pair = src.clamp(min=0)
    grad = (dy[pair // case["K"]] * s["weights"].reshape(-1)[pair].unsqueeze(1)).to(t)
    if s["out"] is not None:
        grad = torch.where((src >= 0).unsqueeze(1), grad, s["out"])
    return {"grad_rows": grad, "grad_weights": torch.where(pos >= 0, dots, torch.zeros_like(dots))}


def plain_int8(s):
    case = s["case"]
    E, K = case["E"], case["K"]
    x = s["x"].float()
    scale = x.abs().amax(1, keepdim=True) / 127.0
    codes = torch.where(scale > 0, x / scale, torch.zeros_like(x)).round().clamp(-127.0, 127.0)
    out = {"codes": codes.to(torch.int8), "scales": scale.squeeze(1)}

    if not E:
        def product(w):
            return codes @ w[0].float().t() * scale * w[1]
    else:
        src = s["sorted_src"].long()
        row = torch.arange(src.numel(), device="cuda")
        expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
        pick = src // K if case["gather"] else row
        if src.numel() <= E:
            # fewer rows than experts: every row with its expert's weights
            def product(w):
                return (w[0][expert].float() * codes[pick].unsqueeze(1)).sum(-1) * w[1][expert] * scale[pick]
        else:
            # every expert's rows side by side, padded to the longest expert's
            most = int(s["counts"].max())
            slot = expert * most + row - s["offsets"].long()[expert]
            a = codes.new_zeros(E * most, case["k"])
            a[slot] = codes[pick]

            def product(w):
                y = torch.bmm(a.view(E, most, -1), w[0].float().mT.contiguous()) * w[1].unsqueeze(1)
                return y.view(E * most, -1)[slot] * scale[pick]
    y = product(s["w"])
    if case["swiglu"]:
        y = y / (1.0 + torch.exp(-y)) * product(s["w_up"])
    out["y"] = y.bfloat16()
    return out


# ---------------------------------------------------------------- the package's operators
def own_grouping(s):
    import sigmoid_top_routing_router_amd as M
    return M.Grouping(s["counts"], s["offsets"], s["sorted_src"], s["src_pos"])


def as_bytes(pair):
    return pair[0].view(torch.uint8), pair[1]


def own_sort(s):
    import sigmoid_top_routing_router_amd as M
    case = s["case"]
    if case["direction"] == "bwd":
        return {"grad_x": M.permute_backward(s["grad_rows"], own_grouping(s))}
    g = M.group_tokens(s["ids"], case["E"])
    x = as_bytes(s["x"]) if case["rows"] == "e4m3" else s["x"]
    return {"rows": M.permute(x, g, out=s["out"]), "counts": g.counts, "offsets": g.offsets,
            "sorted_src": g.sorted_src, "src_pos": g.src_pos}


def own_back(s):
    import sigmoid_top_routing_router_amd as M
    case = s["case"]
    if case["direction"] == "fwd":
        y, kept = M.unpermute(s["expert_rows"], own_grouping(s), weights=s["weights"],
                              base=s["base"], checkpoint=case["kept"])
        out = {"y": y}
        if case["kept"]:
            out["codes"], out["scales"] = kept[0].view(torch.float8_e4m3fn), kept[1]
        return out
    rows = as_bytes(s["expert_rows"]) if case["kept"] else s["expert_rows"]
    grad, dw = M.unpermute_backward(s["grad_y"], own_grouping(s), weights=s["weights"], rows=rows,
                                    out=s["out"])
    return {"grad_rows": grad, "grad_weights": dw}


def own_int8(s):
    import sigmoid_top_routing_router_amd as M
    case = s["case"]
    q = M.int8_quantize_rows(s["x"])
    y = M.int8_matmul(q, s["w"], w_up=s["w_up"], grouping=own_grouping(s) if case["E"] else None,
                      gather=case["gather"])
    return {"codes": q[0], "scales": q[1], "y": y}


PLAIN = {"sort": plain_sort, "back": plain_back, "int8": plain_int8}
OWN = {"sort": own_sort, "back": own_back, "int8": own_int8}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "int8":
        N, k, cols, E, K = (case[n] for n in ("N", "k", "cols", "E", "K"))
        tokens = N if case["gather"] or not E else N * K
        rows = N * K if E else N
        # the weights of the experts that are used, with their channels' scales
        used = E * (1.0 - (1.0 - K / E) ** N) if E else 1
        moved = tokens * (3 * k + 4) + used * (2 if case["swiglu"] else 1) * cols * (k + 4)
        moved += rows * cols * 2 + (rows * 4 + E * 4 if E else 0)
        return {"bytes": int(moved), "flops": 2 * rows * k * cols * (2 if case["swiglu"] else 1)}
    N, d, E, K = (case[n] for n in ("N", "d", "E", "K"))
    size = 4 if case["rows"] == "f32" else 2
    kept = d + d // GROUP * 4  # a row in 8 bits
    # pairs whose expert is here
    pairs = N * K // 2 if case["away"] else N * K
    if case["op"] == "sort":
        if case["direction"] == "bwd":
            return {"bytes": pairs * d * size + N * d * size + N * K * 4, "flops": pairs * d}
        token = kept if case["rows"] == "e4m3" else d * size
        return {"bytes": N * token + pairs * d * size + 3 * N * K * 4 + E * 8, "flops": pairs * d}
    if case["direction"] == "fwd":
        moved = pairs * d * size + N * d * size * (2 if case["base"] else 1) + N * K * 4
        moved += (N * K * 4 if case["weights"] else 0) + (pairs * kept if case["kept"] else 0)
        return {"bytes": moved, "flops": 2 * pairs * d}
    moved = N * d * size + pairs * (kept if case["kept"] else d * size) + pairs * d * size
    return {"bytes": moved + N * K * 12, "flops": 3 * pairs * d}


# ---------------------------------------------------------------- from the definitions, 64 bits
def exact_group(ids, E):
    flat = ids.reshape(-1).long()
    here = ((flat >= 0) & (flat < E)).nonzero().squeeze(1)
    # expert first, then the pair: one number each
    pairs = torch.sort(flat[here] * flat.numel() + here).values % flat.numel()
    counts = torch.bincount(flat[here], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    sorted_src = torch.full_like(flat, -1, dtype=torch.int32)
    sorted_src[:pairs.numel()] = pairs.int()
    src_pos = torch.full_like(sorted_src, -1)
    src_pos[pairs] = torch.arange(pairs.numel(), dtype=torch.int32, device="cuda")
    return {"counts": counts.int(), "offsets": offsets, "sorted_src": sorted_src,
            "src_pos": src_pos.view(ids.shape)}


def exact_kept(pair):
    return pair[0].double() * pair[1].double().repeat_interleave(GROUP, 1)


def exact_rows(s, case):
    K, n = case["K"], int(s["offsets"][-1])
    pairs = s["sorted_src"][:n].long()
    token = torch.div(pairs, K, rounding_mode="floor")

    def sized(rows):
        """The rows that are sorted; behind them what the buffer held."""
        return torch.cat([rows, rows.new_zeros(case["N"] * K - n, rows.shape[1])])

    if case["op"] == "sort":
        if case["direction"] == "bwd":
            total = torch.zeros(case["N"], case["d"], dtype=torch.float64, device="cuda")
            return {"grad_x": total.index_add_(0, token, s["grad_rows"][:n].double())}
        out = exact_group(s["ids"], case["E"])
        x = exact_kept(s["x"]) if case["rows"] == "e4m3" else s["x"].double()
        out["rows"] = sized(x.index_select(0, token))
        return out
    w = None if s["weights"] is None else s["weights"].double().flatten()[pairs].unsqueeze(1)
    if case["direction"] == "fwd":
        rows = s["expert_rows"].double()
        y = torch.zeros(case["N"], case["d"], dtype=torch.float64, device="cuda")
        if s["base"] is not None:
            y += s["base"].double()
        y.index_add_(0, token, rows[:n] if w is None else rows[:n] * w)
        out = {"y": y}
        if case["kept"]:
            blocks = rows.unflatten(1, (-1, GROUP))
            top = torch.maximum(blocks.amax(2), -blocks.amin(2)) / E4M3_MAX
            out["scales"] = top
            out["codes"] = (blocks / top.unsqueeze(2)).flatten(1)  # before the rounding to E4M3
        return out
    rows = exact_kept(s["expert_rows"]) if case["kept"] else s["expert_rows"].double()
    dy = s["grad_y"].double().index_select(0, token)
    dw = torch.zeros(case["N"] * K, dtype=torch.float64, device="cuda")
    dw[pairs] = torch.einsum("pd,pd->p", rows[:n], dy)
    return {"grad_rows": sized(dy * w), "grad_weights": dw.view(case["N"], K)}


def exact_int8(s, case):
    x = s["x"].double()
    top = torch.linalg.vector_norm(x, ord=float("inf"), dim=1, keepdim=True)
    codes = torch.round(x * (127.0 / torch.where(top == 0, torch.ones_like(top), top)))
    # half of the largest value lies between two integers: which one it gets goes
    # by the rounding of the scale
    out = {"codes": None, "scales": (top / 127.0).squeeze(1)}
    values = codes * (top / 127.0)

    def dense(rows, e):
        def weight(w):
            codes, scale = (w[0], w[1]) if e is None else (w[0][e], w[1][e])
            return codes.double() * scale.double().unsqueeze(1)
        y = rows @ weight(s["w"]).t()
        return torch.nn.functional.silu(y) * (rows @ weight(s["w_up"]).t()) if case["swiglu"] else y

    if not case["E"]:
        out["y"] = dense(values, None)
        return out
    out["y"] = torch.empty(s["sorted_src"].numel(), case["cols"], dtype=torch.float64, device="cuda")
    edge = s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = edge[e], edge[e + 1]
        if hi > lo:
            pick = s["sorted_src"][lo:hi].long() // case["K"] if case["gather"] else slice(lo, hi)
            out["y"][lo:hi] = dense(values[pick], e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return exact_int8(s, case) if case["op"] == "int8" else exact_rows(s, case)

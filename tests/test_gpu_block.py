"""The operators of a block run together, as a training step and a serving step
use them: rms_norm -> forward -> balance_loss, and back through
balance_loss_backward, lei_backward, backward and rms_norm_backward; and
rms_norm(quantize) -> forward_fp8(x_quant).

Tolerances of the step, pooled (relative L2).  A bf16 rounding is off by at
most half a step, 2^-8 / sqrt(3) rms, and roundings are independent.  The
gradients are compared with the fp64 block's at the same inputs and the same
selection.  On the way to grad of the sublayer's output: the normed rows y
(which reach G, U and through them H, silu' and every product: gain 2, twice),
dG / dU / s H, grad_x and the result: sqrt(4 + 4 + 1 + 1 + 1) < 3.4 of
2^-8 / sqrt(3), below 2 * 2^-8; a weight's gradient has fewer."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests.gpu_util import (Y_REL_L2_FP8_TOKEN, bf16_dev, check_output, dev, host, rel_l2, say)
from tests.test_gpu_backward import bf16, f64

pytestmark = pytest.mark.gpu

EPS = 1e-6
COEF = 1e-2
LAM, TAU = 1e-3, 2.0
STEP = 2 * 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def block(seed, N, d, E, K, h, hs):
    rng = np.random.default_rng(seed)
    P = dict(sub=bf16(rng, 0.7, N, d), dy=bf16(rng, 0.05, N, d),
             w=O.f32_to_bf16_rne((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)),
             post=O.f32_to_bf16_rne((0.5 + 0.1 * rng.standard_normal(d)).astype(np.float32)),
             w_router=bf16(rng, 1.5 * d ** -0.5, E, d), w_gate=bf16(rng, d ** -0.5, E, h, d),
             w_up=bf16(rng, d ** -0.5, E, h, d), w_down=bf16(rng, h ** -0.5, E, d, h))
    if hs:
        P.update(ws_gate=bf16(rng, d ** -0.5, 1, hs, d), ws_up=bf16(rng, d ** -0.5, 1, hs, d),
                 ws_down=bf16(rng, hs ** -0.5, 1, d, hs))
    P["stream"] = (2.0 * rng.standard_normal((N, d))).astype(np.float32)
    P["dstream"] = (0.05 * rng.standard_normal((N, d))).astype(np.float32)
    return P


def to_dev(M, P):
    T = {k: bf16_dev(v) if v.dtype == np.uint16 else dev(v) for k, v in P.items()}
    W = M.ExpertWeights(**{k: v for k, v in T.items() if k.startswith("w_") or k.startswith("ws_")})
    return T, W


def step(M, T, W, K, cu):
    """One training step of the block around the layer."""
    y, r, _ = M.rms_norm(T["sub"], T["w"], EPS, T["stream"], T["post"])
    out, aux = M.forward(y, W, K, aux=("logits", "topk_ids"))
    Z, ids = aux["logits"], aux["topk_ids"]
    loss, counts, _ = M.balance_loss(Z, ids, COEF, segments=cu)
    _, dz, _ = M.lei_backward(ids, Z.shape[1], Z, lam=LAM, tau=TAU, scores_out=False)
    dz = M.balance_loss_backward(Z, counts, COEF, segments=cu, grad_logits=dz, inplace=True)
    dx, dz, G = M.backward(T["dy"], y, W, Z, ids, dz, inplace=True)
    dsub, dstream, dw, dpost = M.rms_norm_backward(dx, r, T["w"], EPS, T["dstream"], T["sub"],
                                                   T["post"])
    return dict(out=out, Z=Z, ids=ids, loss=loss, logits=dz, sub=dsub, stream=dstream, w=dw,
                post=dpost, **{k: getattr(G, k) for k in T if k.startswith(("w_", "ws_"))})


def silu(g):
    return g / (1.0 + np.exp(-g))


def plain_forward(f, ids, spans, counts, lei):
    """The scalar that the step differentiates, in fp64: dy . layer(y) +
    dstream . r + the balance loss + the injection's term, with the selection
    and the loads held."""
    r, y, _ = B.rms_norm(f["sub"], f["w"], EPS, f["stream"], f["post"])
    Z = y @ f["w_router"].T
    S = 1.0 / (1.0 + np.exp(-Z))
    total = float((f["dstream"] * r).sum()) + float((S * lei).sum())
    total += B.balance_loss(Z, counts, COEF, "sigmoid_norm", spans)[0]
    out = np.zeros_like(y)
    for e in range(Z.shape[1]):
        t, k = np.nonzero(ids == e)
        if len(t):
            H = silu(y[t] @ f["w_gate"][e].T) * (y[t] @ f["w_up"][e].T)
            np.add.at(out, t, S[t, e][:, None] * (H @ f["w_down"][e].T))
    if "ws_gate" in f:
        out += (silu(y @ f["ws_gate"][0].T) * (y @ f["ws_up"][0].T)) @ f["ws_down"][0].T
    return total + float((f["dy"] * out).sum())


def plain_gradients(f, ids, spans, counts, lei):
    r, y, _ = B.rms_norm(f["sub"], f["w"], EPS, f["stream"], f["post"])
    Z = y @ f["w_router"].T
    s = 1.0 / (1.0 + np.exp(-Z))
    dz = B.balance_loss_backward(Z, counts, COEF, "sigmoid_norm", spans)[0] + lei * s * (1 - s)
    shared = (f["ws_gate"][0], f["ws_up"][0], f["ws_down"][0]) if "ws_gate" in f else None
    G, _ = B.layer_backward(y, f["dy"], Z, ids, f["w_router"], f["w_gate"], f["w_up"], f["w_down"],
                            shared, dz)
    dsub, dr, dw, dp = B.rms_norm_backward(G["x"], r, f["w"], EPS, f["dstream"], f["sub"], f["post"])
    return dict(G, sub=dsub, stream=dr, w=dw, post=dp)


SHAPES = [(700, 320, 24, 3, 96, 160), (257, 128, 9, 8, 64, 0), (65, 2560, 12, 2, 128, 64)]


@pytest.mark.parametrize("N,d,E,K,h,hs", SHAPES)
def test_training_step(M, N, d, E, K, h, hs):
    say("block step", N, d, E, K, h, hs)
    P = block(N + d, N, d, E, K, h, hs)
    T, W = to_dev(M, P)
    cuts = [0, N // 3, N // 3, N - 5, N]                 # an empty segment among them
    got = step(M, T, W, K, dev(np.array(cuts, np.int32)))
    spans = list(zip(cuts[:-1], cuts[1:]))
    ids = host(got["ids"])
    counts = B.segment_counts(ids, E, spans)
    _, _, _, lei = O.lei_injection(ids, E, LAM, TAU)
    f = {k: (O.bf16_to_f32(v) if v.dtype == np.uint16 else v).astype(np.float64)
         for k, v in P.items()}
    want = plain_gradients(f, ids, spans, counts, lei)
    for k in ("logits", "sub", "stream", "w", "post", *[k for k in P if k.startswith(("w_", "ws_"))]):
        e = rel_l2(f64(got[k]).reshape(want[k].shape), want[k])
        say(k, f"{e:.2e}")
        assert e <= STEP, (k, e)
    # the plain gradients themselves, against differences of the plain step: a
    # central difference at eps is off by eps^2 of the third derivative and
    # 2^-52 / eps of the value's terms
    rng = np.random.default_rng(3)
    for k in ("sub", "w", "post", "stream", "w_router", "w_gate"):
        v = rng.standard_normal(f[k].shape)
        v *= np.linalg.norm(f[k]) / np.linalg.norm(v)
        eps = 1e-5
        hi = plain_forward({**f, k: f[k] + eps * v}, ids, spans, counts, lei)
        lo = plain_forward({**f, k: f[k] - eps * v}, ids, spans, counts, lei)
        line = float((want[k] * v).sum())
        size = float(np.linalg.norm(want[k]) * np.linalg.norm(v))
        assert abs((hi - lo) / (2 * eps) - line) <= 1e-6 * size, k


def test_training_step_captured(M):
    """The whole step in a graph, replayed on new inputs in its buffers, with
    eager steps between: every replay gives the eager bits."""
    import torch
    N, d, E, K, h, hs = SHAPES[0]
    say("block step graph")
    T, W = to_dev(M, block(1, N, d, E, K, h, hs))
    cu = dev(np.array([0, 100, N], np.int32))
    step(M, T, W, K, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(M, T, W, K, cu)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            cap = step(M, T, W, K, cu)
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        other = block(seed, N, d, E, K, h, hs)
        for k in ("sub", "dy", "stream", "dstream"):
            T[k].copy_(bf16_dev(other[k]) if other[k].dtype == np.uint16 else dev(other[k]))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = {k: v.clone() for k, v in cap.items()}
        eager = step(M, T, W, K, cu)
        torch.cuda.synchronize()
        for k, v in eager.items():
            assert torch.equal(v, replayed[k]), (seed, k)


# ---------------------------------------------------------------- E4M3 serving
def fp8_layer(M, seed, E, K, d, h, hs, packed):
    rng = np.random.default_rng(seed)
    w = dict(w_router=bf16(rng, 1.5 * d ** -0.5, E, d), w_gate=bf16(rng, d ** -0.5, E, h, d),
             w_up=bf16(rng, d ** -0.5, E, h, d), w_down=bf16(rng, h ** -0.5, E, d, h))
    if hs:
        w.update(ws_gate=bf16(rng, d ** -0.5, 1, hs, d), ws_up=bf16(rng, d ** -0.5, 1, hs, d),
                 ws_down=bf16(rng, hs ** -0.5, 1, d, hs))
    W = M.quantize_experts(M.ExpertWeights(**{k: bf16_dev(v) for k, v in w.items()}))
    return w, M.pack_gateup(W) if packed else W


@pytest.mark.parametrize("N,hs,packed", [(1, 0, False), (1, 256, False), (40, 256, False),
                                         (64, 128, True), (65, 256, True), (700, 256, False)])
def test_given_codes_of_x_are_the_layers_own(M, N, hs, packed):
    import torch
    say("fp8 layer, codes given", N, hs, packed)
    E, K, d, h = 16, 4, 384, 256
    _, W = fp8_layer(M, N, E, K, d, h, hs, packed)
    x = bf16_dev(bf16(np.random.default_rng(N), 1.0, N, d))
    y0, a0 = M.forward_fp8(x, W, K, aux=("logits", "topk_ids"))
    q = M.fp8_quantize_rows(x)
    y1, a1 = M.forward_fp8(x, W, K, aux=("logits", "topk_ids"), x_quant=q)
    assert torch.equal(y0, y1) and torch.equal(a0["logits"], a1["logits"])
    # the logits given: x is not read
    y2 = M.forward_fp8(torch.full_like(x, float("nan")), W, K, logits_in=a0["logits"], x_quant=q)
    y3 = M.forward_fp8(x, W, K, logits_in=a0["logits"])
    assert torch.equal(y2, y3)


@pytest.mark.parametrize("N", [1, 33, 300])
def test_serving_step(M, N):
    """The norm's codes straight into the layer, against the oracle's layer on
    the same codes; the bf16 copy goes to the router only."""
    import torch
    say("norm into the fp8 layer", N)
    E, K, d, h, hs = 12, 3, 256, 128, 128
    w, W = fp8_layer(M, 50, E, K, d, h, hs, False)
    rng = np.random.default_rng(N)
    sub, wn = bf16_dev(bf16(rng, 0.8, N, d)), bf16_dev(O.f32_to_bf16_rne(np.ones(d, np.float32)))
    stream = dev((2 * rng.standard_normal((N, d))).astype(np.float32))

    def serve():
        y, r, q = M.rms_norm(sub, wn, EPS, stream, quantize=True)
        out, aux = M.forward_fp8(y, W, K, aux=("topk_ids", "topk_weights"), x_quant=q)
        return y, q, out, aux
    y, q, out, aux = serve()
    codes, scales = host(q[0]), host(q[1])
    ids, S = host(aux["topk_ids"]), host(aux["topk_weights"]).astype(np.float64)
    c = {k: host(getattr(W, k)) for k in ("w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down",
                                          "ws_gate", "ss_gate", "ws_up", "ss_up", "ws_down",
                                          "ss_down")}
    ref = O.swiglu_fp8(codes, scales, c["ws_gate"][0], c["ss_gate"][0], c["ws_up"][0],
                       c["ss_up"][0], c["ws_down"][0], c["ss_down"][0])
    for e in range(E):
        t, k = np.nonzero(ids == e)
        if len(t):
            ref[t] += S[t, k][:, None] * O.swiglu_fp8(
                codes[t], scales[t], c["w_gate"][e], c["s_gate"][e], c["w_up"][e], c["s_up"][e],
                c["w_down"][e], c["s_down"][e])
    check_output(f64(out), ref, "serving step", Y_REL_L2_FP8_TOKEN)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        serve()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            cap = serve()
    for rep in range(3):
        stream.add_(0.25)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        held = cap[2].clone()
        assert torch.equal(held, serve()[2]), rep
        torch.cuda.synchronize()


def test_given_codes_refusals(M):
    E, K, d, h = 8, 2, 256, 128
    _, W = fp8_layer(M, 3, E, K, d, h, 0, False)
    x = bf16_dev(bf16(np.random.default_rng(3), 1.0, 5, d))
    codes, scales = M.fp8_quantize_rows(x)
    with pytest.raises(ValueError):
        M.forward_fp8(x, W, K, x_quant=(codes[:4], scales))
    with pytest.raises(TypeError):
        M.forward_fp8(x, W, K, x_quant=(codes, scales.double()))
    with pytest.raises(TypeError):
        M.forward_fp8(x, W, K, x_quant=(codes.cpu(), scales))

"""GPU parity of moe_backward against the plain fp64 form.

Tolerances, worst case per value.  A bf16 rounding is half a step, B = 2^-8
relative.  Weight gradients: one operand (dG, dU, s H or grad_logits_out) is
rounded once and the result once: B mag + B |out|, mag being the product of
the operands' absolute values.  grad_x: the same two (its bound here holds one
rounding of the parts more): 2 B mag + B |out|.  fp32 accumulation: an MFMA
adds 16 products, so a sum over k has at most k / 16 + 20 roundings of 2^-24
of at most mag each: C below, with k the longest sum of the path.
grad_logits: Q, G and U each within C of their terms, H and Q . H a few more
roundings (2^-18 together with sigma): (C + 2^-18) mag, plus the rounding of
the sum.  Pooled, errors are independent: a half step is at most B / sqrt(3)
rms, two of them (or three) below or at B."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests.gpu_util import bf16_dev, dev, host, rel_l2, say

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def bf16(rng, std, *shape):
    return O.f32_to_bf16_rne(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def make(seed, N, d, E, K, h, hs, ids=None, router=True):
    rng = np.random.default_rng(seed)
    L = dict(x=bf16(rng, 1.0, N, d), dy=bf16(rng, 0.05, N, d),
             w_gate=bf16(rng, d ** -0.5, E, h, d), w_up=bf16(rng, d ** -0.5, E, h, d),
             w_down=bf16(rng, h ** -0.5, E, d, h))
    if router:
        L["w_router"] = bf16(rng, 1.5 * d ** -0.5, E, d)
    if hs:
        L.update(ws_gate=bf16(rng, d ** -0.5, 1, hs, d), ws_up=bf16(rng, d ** -0.5, 1, hs, d),
                 ws_down=bf16(rng, hs ** -0.5, 1, d, hs))
    Z = (1.5 * rng.standard_normal((N, E))).astype(np.float32)
    if ids is None:
        ids = np.argsort(-Z, axis=1, kind="stable")[:, :K]
    return L, Z, np.ascontiguousarray(ids, dtype=np.int32)


def run(M, L, Z, ids, grad=None, **kw):
    W = M.ExpertWeights(**{"w_router": None,
                           **{k: bf16_dev(v) for k, v in L.items() if k.startswith("w")}})
    return M.backward(bf16_dev(L["dy"]), bf16_dev(L["x"]), W, dev(Z), dev(ids),
                      grad_logits=None if grad is None else dev(grad), **kw)


def f64(t):
    a = host(t)
    return (O.bf16_to_f32(a) if a.dtype == np.uint16 else a).astype(np.float64)


def check(L, Z, ids, got, grad=None, pooled=True):
    dx, dz, G = got
    f = {k: O.bf16_to_f32(v) for k, v in L.items()}
    shared = (f["ws_gate"][0], f["ws_up"][0], f["ws_down"][0]) if "ws_gate" in f else None
    want, mag = B.layer_backward(f["x"], f["dy"], Z, ids, f.get("w_router"), f["w_gate"], f["w_up"],
                                 f["w_down"], shared, grad)
    N, d = f["x"].shape
    longest = max(N, d, f["w_gate"].shape[1], Z.shape[1], 0 if shared is None else shared[0].shape[0])
    c = (longest / 16 + 20) * 2.0 ** -24
    z = f64(dz)
    err = np.abs(z - want["logits"])
    assert np.all(err <= (c + 2.0 ** -18) * mag["logits"] + 2.0 ** -24 * np.abs(want["logits"]) + 1e-37)
    out = {"x": f64(dx), **{k: f64(getattr(G, k)) for k in L if k.startswith("w")}}
    for k, v in out.items():
        rounded = 2 if k == "x" else 1
        tol = (rounded * HALF * 1.01 + 2 * c + 2.0 ** -17) * mag[k] + HALF * np.abs(want[k]) + 1e-37
        bad = np.abs(v - want[k]) > tol
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[:3].tolist())
        if pooled and v.size > 4096:
            e = rel_l2(v, want[k])
            say(k, f"{e:.2e}")
            assert e <= HALF, (k, e)
    for k in ("w_router", "ws_gate", "ws_up", "ws_down"):
        assert (getattr(G, k) is None) == (k not in L)
    return want


@pytest.mark.parametrize("N,d,E,K,h,hs", [
    (1, 64, 9, 8, 32, 0), (5, 64, 3, 2, 32, 64), (65, 128, 8, 2, 96, 32),
    (333, 320, 20, 4, 160, 0), (300, 192, 7, 1, 288, 160), (700, 512, 12, 3, 256, 256),
    (257, 576, 65, 6, 64, 128), (130, 2560, 10, 2, 64, 0), (40, 64, 384, 6, 32, 32),
    (90, 128, 5, 2, 768, 96)])
def test_parity(M, N, d, E, K, h, hs):
    say("backward", N, d, E, K, h, hs)
    L, Z, ids = make(N + d + E, N, d, E, K, h, hs)
    check(L, Z, ids, run(M, L, Z, ids))


@pytest.mark.parametrize("counts", [
    (256, 0, 257, 288), (289, 1, 0, 512), (0, 0, 600, 0), (513, 544, 545, 3)])
def test_segment_lengths(M, counts):
    """Experts without rows, and segments at the tiles' edges."""
    say("backward, segments", counts)
    ids = np.repeat(np.arange(4), counts)[:, None]
    rng = np.random.default_rng(sum(counts))
    ids = ids[rng.permutation(len(ids))]
    L, Z, ids = make(17, len(ids), 128, 4, 1, 64, 0, ids=ids)
    got = run(M, L, Z, ids)
    check(L, Z, ids, got)
    for e, n in enumerate(counts):
        if n == 0:
            assert not f64(got[2].w_gate)[e].any() and not f64(got[2].w_down)[e].any()


def test_long_segment(M):
    """An expert with more rows than the row-offset table of a block holds."""
    say("backward, 9,000 rows in one segment")
    ids = np.zeros((9000, 1), np.int32)
    ids[::100] = 2
    L, Z, ids = make(18, 9000, 64, 4, 1, 32, 32, ids=ids)
    check(L, Z, ids, run(M, L, Z, ids))


def test_added_gradient_inplace_and_no_router(M):
    import torch
    L, Z, ids = make(19, 200, 128, 33, 3, 64, 64)
    grad = (1e-2 * np.random.default_rng(2).standard_normal(Z.shape)).astype(np.float32)
    say("backward, added gradient")
    got = run(M, L, Z, ids, grad)
    check(L, Z, ids, got, grad)
    W = M.ExpertWeights(**{k: bf16_dev(v) for k, v in L.items() if k.startswith("w")})
    g = dev(grad)
    again = M.backward(bf16_dev(L["dy"]), bf16_dev(L["x"]), W, dev(Z), dev(ids), grad_logits=g,
                       inplace=True)
    assert again[1] is g and torch.equal(g, got[1]) and torch.equal(again[0], got[0])
    say("backward, no router")
    L, Z, ids = make(20, 100, 64, 6, 2, 32, 0, router=False)
    check(L, Z, ids, run(M, L, Z, ids))


def test_ids_outside_and_twice(M):
    """A pair with an id outside [0, E) has no gradient; the same id twice in a
    row counts twice."""
    L, Z, ids = make(21, 150, 128, 10, 3, 64, 32)
    ids[::4, 1] = -1
    ids[1::4, 0] = 10
    ids[2::4, 2] = ids[2::4, 0]
    ids[3] = -7
    say("backward, ids outside the range")
    f = {k: O.bf16_to_f32(v) for k, v in L.items()}
    assert f["x"].shape == (150, 128)
    check(L, Z, ids, run(M, L, Z, ids))


def test_padded_rows_that_hold_nan(M):
    """Rows with no expert, NaN and infinities in their x, dy and logits, at the
    start, inside and at the end: the other gradients are the bits of the
    batch with zeros there, and theirs are zeros."""
    import torch
    L, Z, ids = make(25, 300, 128, 6, 2, 96, 0, router=False)
    pad = np.r_[0:9, 100:140, 290:300]
    ids[pad] = -1
    for k in ("x", "dy"):
        L[k][pad] = 0
    Z[pad] = 0
    say("backward, padded rows")
    want = run(M, L, Z, ids)
    check(L, Z, ids, want)
    for k in ("x", "dy"):
        L[k][pad] = 0x7FC0                               # NaN
        L[k][pad[::3]] = 0x7F80                          # inf
    Z[pad] = np.nan
    got = run(M, L, Z, ids)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not got[0][torch.from_numpy(pad).cuda()].any()
    for k in ("w_gate", "w_up", "w_down"):
        assert torch.equal(getattr(got[2], k), getattr(want[2], k)), k


def test_hidden_rows_past_four_gigabytes(M):
    """60,000 x 8 pairs of 2,080: the hidden rows take 6 GB, Q 4.  The last
    expert's gradients and the last tokens' grad_x against fp64."""
    import torch
    N, d, E, K, h = 60000, 64, 9, 8, 2080
    L, Z, ids = make(26, N, d, E, K, h, 0, router=False)
    say("backward, hidden rows past 4 GB")
    dx, dz, G = run(M, L, Z, ids)
    x, dy = (bf16_dev(L[k]).double() for k in ("x", "dy"))
    wg, wu, wd = (bf16_dev(L[k]).double() for k in ("w_gate", "w_up", "w_down"))
    z, sel = dev(Z).double(), dev(ids)

    def pairs(t, e):
        s = torch.sigmoid(z[t, e])[:, None]
        g, u, q = x[t] @ wg[e].t(), x[t] @ wu[e].t(), dy[t] @ wd[e]
        sg = torch.sigmoid(g)
        return s * q * u * sg * (1 + g * (1 - sg)), s * q * g * sg, s * g * sg * u
    c = (N / 16 + 20) * 2.0 ** -24
    e = E - 1
    t = (sel == e).any(dim=1).nonzero()[:, 0]
    dg, du, sh = pairs(t, e)
    for got, a, b in ((G.w_gate, dg, x[t]), (G.w_up, du, x[t]), (G.w_down, dy[t], sh)):
        want, mag = a.t() @ b, a.abs().t() @ b.abs()
        tol = (HALF * 1.01 + 2 * c + 2.0 ** -17) * mag + HALF * want.abs()
        assert bool(((got[e].double() - want).abs() <= tol).all())
        assert float((got[e].double() - want).norm() / want.norm()) <= HALF
    tail = torch.arange(N - 40, N, device="cuda")
    want, mag = torch.zeros(40, d, dtype=torch.float64, device="cuda"), 0.0
    for e in range(E):
        on = (sel[tail] == e).any(dim=1)[:, None]
        dg, du, _ = pairs(tail, e)
        want += on * (dg @ wg[e] + du @ wu[e])
        mag = mag + on * (dg.abs() @ wg[e].abs() + du.abs() @ wu[e].abs())
    tol = (HALF * 1.01 + 2 * c + 2.0 ** -17) * mag + HALF * want.abs()
    assert bool(((dx[tail].double() - want).abs() <= tol).all())


def test_agrees_with_the_forward_pass(M):
    """Differences of the layer's own output: dy . (y(x + v) - y(x - v)) / 2 for
    a direction v, with the selection held by a bias.  y leaves in bf16, so the
    difference is good to the rounding of 2 N d values of y, each half a step
    and independent: std <= |y| 2^-8 / sqrt(3) * |dy| * sqrt(N d) / 2 * sqrt(2)."""
    import torch
    N, d, E, K, h = 64, 256, 8, 2, 64
    L, _, _ = make(22, N, d, E, K, h, 64)
    W = M.ExpertWeights(**{k: bf16_dev(v) for k, v in L.items() if k.startswith("w")})
    x = bf16_dev(L["x"])
    say("backward against differences of forward")
    beta = torch.zeros(E, device="cuda")
    beta[:K] = 100.0                                     # the same experts for every token
    y, aux = M.forward(x, W, K, beta_in=beta, aux=("logits", "topk_ids"))
    dy = bf16_dev(L["dy"])
    dx, _, _ = M.backward(dy, x, W, aux["logits"], aux["topk_ids"])
    # a direction with exact bf16 end points: x (1 + 1/8) and x (1 - 1/8) do not
    # round alike, so take the end points first and their true difference
    hi, lo = (x.float() * 1.0625).bfloat16(), (x.float() * 0.9375).bfloat16()
    step = (hi.double() - lo.double()) / 2
    yh, yl = M.forward(hi, W, K, beta_in=beta), M.forward(lo, W, K, beta_in=beta)
    diff = float((dy.double() * (yh.double() - yl.double())).sum() / 2)
    line = float((dx.double() * step).sum())
    noise = float((dy.double() * y.double()).norm()) * 2.0 ** -8 / 3 ** 0.5 * 2 ** 0.5 / 2
    # third-order term of a function of x along x: bounded by (1/16)^2 of the
    # first-order size, taken as |dy . y|'s spread, the layer being near
    # quadratic in x
    size = float((dy.double() * y.double()).norm())
    assert abs(diff - line) <= 4 * noise + (1 / 16) ** 2 * 4 * size, (diff, line, noise, size)


def test_repeats_stream_and_graph(M):
    import torch
    L, Z, ids = make(23, 1500, 512, 16, 4, 128, 128)
    say("backward graph")
    W = M.ExpertWeights(**{k: bf16_dev(v) for k, v in L.items() if k.startswith("w")})
    dy, x, z, i = bf16_dev(L["dy"]), bf16_dev(L["x"]), dev(Z), dev(ids)
    ws = torch.empty(M.backward_workspace_bytes(1500, 512, 16, 4, 128, 1, 128), dtype=torch.uint8,
                     device="cuda")

    def flat(r):
        return [r[0], r[1]] + [getattr(r[2], k) for k in L if k.startswith("w")]
    ref = flat(M.backward(dy, x, W, z, i))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws.fill_(0xFF)                                       # NaN patterns in the workspace
    torch.cuda.synchronize()
    out = flat(M.backward(dy, x, W, z, i, workspace=ws, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            cap = flat(M.backward(dy, x, W, z, i, workspace=ws))
    for rep in range(3):
        for t in cap:
            t.zero_()
        ws.fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, cap)), rep
        M.backward(dy, x, W, z, i)
        torch.cuda.synchronize()


def test_refusals(M):
    L, Z, ids = make(24, 30, 64, 6, 2, 32, 0)
    W = M.ExpertWeights(**{k: bf16_dev(v) for k, v in L.items() if k.startswith("w")})
    dy, x, z, i = bf16_dev(L["dy"]), bf16_dev(L["x"]), dev(Z), dev(ids)
    say("backward refusals")
    with pytest.raises(ValueError):
        M.backward(dy, x, M.pack_gateup(W), z, i)
    with pytest.raises(ValueError):
        M.backward(dy[:20].contiguous(), x, W, z, i)
    with pytest.raises(ValueError):
        M.backward(dy, x, W, z, i[:20].contiguous())
    with pytest.raises(ValueError):
        M.backward(dy, x, W, z, i, inplace=True)
    with pytest.raises(TypeError):
        M.backward(dy.float(), x, W, z, i)
    with pytest.raises(M.MoeError):
        M.backward(dy, x, W, z, i, workspace=z.view(-1)[:64])

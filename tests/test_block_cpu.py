"""The operators around the layer on the CPU: their entry points size
workspaces and refuse bad arguments before any HIP call, and the plain fp64
gradients agree with differences of the plain fp64 functions."""
import ctypes as C
import os

import numpy as np
import pytest

from oracle import block_oracle as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sigmoid_top_routing_router_amd", "libmoe_mi355x.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_router_amd import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def mem():
    """A host buffer's 256-byte aligned address: only ever compared and checked,
    the calls below are all refused."""
    buf = C.create_string_buffer(1 << 20)
    yield (C.cast(buf, C.c_void_p).value + 255) // 256 * 256


@built
def test_rms_norm_refusals(lib, mem):
    base = dict(x=mem, res=None, post=None, w=mem + 4096, n=4, d=128, eps=1e-6, flags=0,
                y=mem + 8192, r=None, codes=None, scales=None)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_rms_norm(*[a[k] for k in ("x", "res", "post", "w", "n", "d", "eps", "flags",
                                                 "y", "r", "codes", "scales")], None)
    assert call(n=-1) == 2 and call(n=(1 << 27) + 1) == 2
    assert call(d=0) == 2 and call(d=8193) == 2
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(flags=4) == 1
    assert call(x=None) == 1 and call(w=None) == 1
    assert call(y=None) == 1                                  # no output at all
    assert call(codes=mem + 16384) == 1                       # codes without scales
    assert call(scales=mem + 16384) == 1
    assert call(codes=mem + 16384, scales=mem + 32768, d=192) == 2
    assert call(codes=mem + 16384 + 8, scales=mem + 32768) == 1
    assert call(codes=mem + 16384, scales=mem + 32768, y=mem + 8194) == 1
    assert call(x=mem + 1) == 1 and call(y=mem + 8193) == 1
    assert call(res=mem + 16386, flags=1) == 1                # fp32 stream, 2-byte aligned
    assert call(w=mem + 4098, flags=2) == 1
    assert call(y=mem) == 1                                   # y is x
    assert call(r=mem, res=mem + 16384) == 1                  # residual_out is x
    assert call(n=0, x=None, w=None) == 0                     # nothing to enqueue
    assert lib.moe_rms_norm(mem, None, None, mem, 4, 128, 1e-6, 0, None, None, None, None,
                            None) == 1
    assert lib.moe_last_error_message() != b""


@built
def test_rms_norm_backward_refusals(lib, mem):
    need = lib.moe_rms_norm_backward_workspace_bytes(4, 128)
    assert need >= 2 * 128 * 4
    for n, d in ((-1, 128), (4, 0), (4, 8193), ((1 << 27) + 1, 128)):
        assert lib.moe_rms_norm_backward_workspace_bytes(n, d) == 0
    base = dict(dy=mem, r=mem + 4096, x=None, dres=None, w=mem + 8192, post=None, n=4, d=128,
                eps=1e-6, flags=0, dx=mem + 12288, dr=None, dw=mem + 16384, dp=None,
                ws=mem + 65536, wsb=need)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_rms_norm_backward(*[a[k] for k in (
            "dy", "r", "x", "dres", "w", "post", "n", "d", "eps", "flags", "dx", "dr", "dw", "dp",
            "ws", "wsb")], None)
    assert call(d=8193) == 2 and call(n=-1) == 2
    assert call(eps=-1e-9) == 1 and call(flags=8) == 1
    assert call(dy=None) == 1 and call(r=None) == 1 and call(w=None) == 1
    assert call(x=mem + 20480) == 1                           # x without post_weight
    assert call(post=mem + 20480) == 1                        # post_weight without x
    assert call(dp=mem + 20480) == 1                          # its gradient without it
    assert call(dx=None, dw=None) == 1
    assert call(dx=mem) == 1                                  # an output is grad_y
    assert call(dy=mem + 1) == 1 and call(dw=mem + 16386) == 1
    assert call(r=mem + 4098, flags=1) == 1
    assert call(ws=mem + 65537) == 1 and call(ws=None) == 1
    assert call(wsb=need - 1) == 3


@built
def test_balance_refusals(lib, mem):
    need = lib.moe_balance_workspace_bytes(40, 8, 3)
    assert need > 0
    for N, E, G in ((0, 8, 1), ((1 << 24) + 1, 8, 1), (4, 1, 1), (4, 385, 1), (4, 8, 0),
                    (4, 8, (1 << 20) + 1)):
        assert lib.moe_balance_workspace_bytes(N, E, G) == 0
    base = dict(z=mem, ids=mem + 4096, cin=None, b=mem + 8192, e=mem + 8448, N=40, E=8, K=2, G=3,
                score=1, coef=1e-2, loss=mem + 12288, cout=mem + 16384, mean=None,
                ws=mem + 65536, wsb=need)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_balance_loss(*[a[k] for k in (
            "z", "ids", "cin", "b", "e", "N", "E", "K", "G", "score", "coef", "loss", "cout",
            "mean", "ws", "wsb")], None)
    assert call(N=0) == 2 and call(E=385) == 2 and call(G=0) == 2
    assert call(K=0) == 2 and call(K=9) == 2 and call(E=2, K=2) == 2
    assert call(b=None) == 1 and call(e=None) == 1
    assert call(b=None, e=None) == 1                          # three segments, no bounds
    assert call(score=3) == 1 and call(score=-1) == 1
    assert call(coef=float("nan")) == 1
    assert call(z=None) == 1 and call(loss=None) == 1
    assert call(ids=None) == 1                                # neither ids nor counts
    assert call(z=mem + 2) == 1 and call(mean=mem + 2) == 1
    assert call(cin=mem + 16384) == 1                         # counts_out is counts_in
    assert call(ws=None) == 1 and call(ws=mem + 65540) == 1
    assert call(wsb=need - 1) == 3

    grad = dict(z=mem, c=mem + 4096, b=mem + 8192, e=mem + 8448, N=40, E=8, G=3, score=1,
                coef=1e-2, gl=None, gin=None, out=mem + 16384)

    def back(**kw):
        a = dict(grad, **kw)
        return lib.moe_balance_loss_backward(*[a[k] for k in (
            "z", "c", "b", "e", "N", "E", "G", "score", "coef", "gl", "gin", "out")], None)
    assert back(N=0) == 2 and back(G=1 << 21) == 2
    assert back(e=None) == 1 and back(score=5) == 1 and back(coef=float("inf")) == 1
    assert back(z=None) == 1 and back(c=None) == 1 and back(out=None) == 1
    assert back(out=mem) == 1                                 # the logits themselves
    assert back(gl=mem + 2) == 1


@built
def test_forward_fp8_quantized_refusals(lib, mem):
    from sigmoid_top_routing_router_amd._lib import MoeFp8Weights, MoeProblem
    p = MoeProblem(N=4, d=128, E=4, K=2, h=128, n_shared=1, h_shared=128, flags=0)
    w = MoeFp8Weights(*([mem] * 13))

    def call(codes=mem, scales=mem, wsb=1 << 30, x=mem):
        return lib.moe_forward_fp8_quantized(C.byref(p), C.byref(w), x, codes, scales, None, mem,
                                             None, mem, wsb, None)
    assert call(codes=None) == 1 and call(scales=None) == 1
    assert call(codes=mem + 8) == 1 and call(scales=mem + 2) == 1
    assert call(x=None) == 1
    assert call(wsb=64) == 3


def _differences(f, x, step):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + step
        hi = f()
        flat[i] = keep - step
        out[i] = (hi - f()) / (2 * step)
        flat[i] = keep
    return g


@pytest.mark.parametrize("post", [False, True])
def test_norm_gradient_formula(post):
    rng = np.random.default_rng(7)
    n, d, eps = 3, 5, 1e-2
    x, res = rng.standard_normal((n, d)), rng.standard_normal((n, d))
    w, pw = rng.standard_normal(d), (rng.standard_normal(d) if post else None)
    dy, dres = rng.standard_normal((n, d)), rng.standard_normal((n, d))

    def value():
        r, y, _ = B.rms_norm(x, w, eps, res, pw)
        return float((y * dy).sum() + (r * dres).sum())

    r = B.rms_norm(x, w, eps, res, pw)[0]
    dx, dr, dw, dp = B.rms_norm_backward(dy, r, w, eps, dres, x if post else None, pw)
    # central differences of step 1e-5: error about 1e-10 times a third
    # derivative of order 10, and 1e-16 / 1e-5 from rounding
    pairs = [(dx, x), (dr, res), (dw, w)] + ([(dp, pw)] if post else [])
    for got, at in pairs:
        assert np.abs(got - _differences(value, at, 1e-5)).max() < 1e-7


@pytest.mark.parametrize("score", ["sigmoid", "sigmoid_norm", "softmax"])
def test_balance_gradient_formula(score):
    rng = np.random.default_rng(11)
    z = rng.standard_normal((7, 6))
    ids = np.argsort(-z, axis=1)[:, :2]
    spans = [(0, 3), (3, 3), (4, 7)]                          # row 3 belongs to none
    counts = B.segment_counts(ids, 6, spans)

    def value():
        return B.balance_loss(z, counts, 0.5, score, spans)[0]

    dz, size = B.balance_loss_backward(z, counts, 0.5, score, spans)
    assert np.abs(dz - _differences(value, z, 1e-5)).max() < 1e-8
    assert np.all(dz[3] == 0) and np.all(np.abs(dz) <= size + 1e-18)


@built
def test_backward_refusals(lib, mem):
    from sigmoid_top_routing_router_amd._lib import MoeGrads, MoeProblem, MoeWeights

    def problem(**kw):
        return MoeProblem(**dict(dict(N=4, d=64, E=4, K=2, h=32, n_shared=1, h_shared=32, flags=0), **kw))
    need = lib.moe_backward_workspace_bytes(C.byref(problem()))
    assert need > 0
    # the routing flags of the forward call are allowed, packed weights are not
    assert lib.moe_backward_workspace_bytes(C.byref(problem(flags=11))) == need
    for bad in (dict(flags=4), dict(flags=16), dict(N=0), dict(K=9), dict(E=2), dict(d=96),
                dict(h=40), dict(n_shared=2), dict(N=1 << 18, d=8192)):
        assert lib.moe_backward_workspace_bytes(C.byref(problem(**bad))) == 0, bad
    # N d of exactly 4 GiB - 128 KiB passes, a row more does not
    rows = (2 ** 32 - 2 ** 17) // (2 * 8192)
    assert lib.moe_backward_workspace_bytes(C.byref(problem(N=rows, d=8192, h=32))) > 0
    assert lib.moe_backward_workspace_bytes(C.byref(problem(N=rows + 1, d=8192, h=32))) == 0
    w = MoeWeights(*([mem] * 7))
    outs = [mem + 4096, mem + 8192] + [mem + 16384] * 7
    base = dict(p=problem(), w=w, x=mem, dy=mem, z=mem, ids=mem, gz=None, g=MoeGrads(*outs),
                ws=mem + 65536, wsb=need)

    def call(**kw):
        a = dict(base, **kw)
        ref = [None if a[k] is None else C.byref(a[k]) for k in ("p", "w", "g")]
        return lib.moe_backward(ref[0], ref[1], a["x"], a["dy"], a["z"], a["ids"], a["gz"], ref[2],
                                a["ws"], a["wsb"], None)

    def grads(i, v):
        return MoeGrads(*[v if j == i else o for j, o in enumerate(outs)])

    def weights(i, v):
        return MoeWeights(*[v if j == i else mem for j in range(7)])
    assert call(p=None) == 2 or call(p=None) == 1
    for name in ("w", "x", "dy", "z", "ids", "g"):
        assert call(**{name: None}) == 1, name
    for i in range(9):
        assert call(g=grads(i, None)) == 1, i                 # every gradient is required
    for i in range(7):
        assert call(w=weights(i, None)) == 1, i               # w_router: its gradient is given
        assert call(w=weights(i, mem + 8)) == 1, i
    assert call(x=mem + 8) == 1 and call(z=mem + 2) == 1 and call(g=grads(3, mem + 8)) == 1
    assert call(g=grads(1, mem)) == 1                         # the logits themselves
    assert call(g=grads(0, mem)) == 1                         # grad_x is x
    assert call(p=problem(flags=4)) == 1
    assert call(ws=None) == 1 and call(ws=mem + 65540) == 1
    assert call(wsb=need - 1) == 3


def test_layer_gradient_formula():
    rng = np.random.default_rng(3)
    N, d, E, K, h, hs = 4, 3, 4, 2, 2, 3
    t = dict(x=rng.standard_normal((N, d)), wr=rng.standard_normal((E, d)),
             wg=rng.standard_normal((E, h, d)), wu=rng.standard_normal((E, h, d)),
             wd=rng.standard_normal((E, d, h)), sg=rng.standard_normal((hs, d)),
             su=rng.standard_normal((hs, d)), sd=rng.standard_normal((d, hs)))
    dy, extra = rng.standard_normal((N, d)), rng.standard_normal((N, E))
    ids = np.argsort(-(t["x"] @ t["wr"].T), axis=1)[:, :K]

    def mlp(x, g, u, w):
        a = x @ g.T
        return (a / (1 + np.exp(-a)) * (x @ u.T)) @ w.T

    def value():
        z = t["x"] @ t["wr"].T
        y = mlp(t["x"], t["sg"], t["su"], t["sd"])
        for i in range(N):
            for e in ids[i]:
                y[i] += mlp(t["x"][i:i + 1], t["wg"][e], t["wu"][e], t["wd"][e])[0] / (1 + np.exp(-z[i, e]))
        return float((y * dy).sum() + (z * extra).sum())

    out, mag = B.layer_backward(t["x"], dy, t["x"] @ t["wr"].T, ids, t["wr"], t["wg"], t["wu"],
                                t["wd"], (t["sg"], t["su"], t["sd"]), extra)
    for name, key in (("x", "x"), ("wr", "w_router"), ("wg", "w_gate"), ("wu", "w_up"),
                      ("wd", "w_down"), ("sg", "ws_gate"), ("su", "ws_up"), ("sd", "ws_down")):
        got = out[key].reshape(t[name].shape)
        assert np.abs(got - _differences(value, t[name], 1e-5)).max() < 1e-6, name
        if key != "x":  # the sizes bound the sums
            assert np.all(np.abs(out[key]) <= mag[key] + 1e-12)


@built
def test_outputs_that_are_one_buffer(lib, mem):
    """Two outputs in one buffer are refused before any HIP call."""
    assert lib.moe_rms_norm(mem, mem + 4096, None, mem + 8192, 4, 128, 1e-6, 0, mem + 12288,
                            mem + 12288, None, None, None) == 1
    need = lib.moe_rms_norm_backward_workspace_bytes(4, 128)
    assert lib.moe_rms_norm_backward(mem, mem + 4096, mem + 20480, None, mem + 8192, mem + 24576,
                                     4, 128, 1e-6, 0, mem + 12288, mem + 12288, None, None,
                                     mem + 65536, need, None) == 1
    assert lib.moe_rms_norm_backward(mem, mem + 4096, mem + 20480, None, mem + 8192, mem + 24576,
                                     4, 128, 1e-6, 0, None, None, mem + 12288, mem + 12288,
                                     mem + 65536, need, None) == 1

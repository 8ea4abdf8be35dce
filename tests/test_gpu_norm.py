"""GPU parity of moe_rms_norm and moe_rms_norm_backward against the plain fp64
forms.

Tolerances.  STAT = 2^-18 bounds the relative error of a reciprocal root mean
square and of a mean over a row in fp32: a thread adds eight squares one after
the other, then six wave steps and at most 16 waves (30 roundings of 2^-24,
halved by the root), the root and two products one to two more each; a gradient
uses two such factors and their products.  The magnitudes it multiplies are the
sums of the absolute terms, so that cancelling terms are covered.  A value that
leaves in bf16 adds half a step, 2^-8 of it; an E4M3 code half of its step,
2^-4 of it or 2^-10 among the subnormals."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu

STAT = 2.0 ** -18
BF16 = 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def f64(t):
    a = host(t)
    return (O.bf16_to_f32(a) if a.dtype == np.uint16 else a).astype(np.float64)


def make(seed, n, d, residual, post, weight, offset=0):
    """Tensors of a case; offset > 0 starts every one that many elements into
    its storage (no 16-byte alignment)."""
    import torch
    rng = np.random.default_rng(seed)

    def t(shape, std, dtype, mean=0.0):
        a = torch.from_numpy((mean + std * rng.standard_normal(shape)).astype(np.float32)).to(dtype)
        flat = torch.empty(a.numel() + offset, dtype=dtype, device="cuda")
        flat[offset:] = a.reshape(-1).cuda()
        return flat[offset:].view(a.shape)
    wt = torch.float32 if weight == "f32" else torch.bfloat16
    st = torch.float32 if residual == "f32" else torch.bfloat16
    s = dict(x=t((n, d), 0.7, torch.bfloat16), w=t((d,), 0.2, wt, 1.0),
             post=t((d,), 0.1, wt, 0.5) if post else None,
             res=None if residual == "none" else t((n, d), 3.0, st),
             dy=t((n, d), 0.01, torch.bfloat16),
             dres=None if residual == "none" else t((n, d), 0.01, st))
    return s


def check_forward(s, y, r, quant):
    x, w, post, res = (None if s[k] is None else f64(s[k]) for k in ("x", "w", "post", "res"))
    rr, yy, a = B.rms_norm(x, w, EPS, res, post)
    u = rr if res is None else rr - res
    mag = np.abs(u) + (0 if res is None else np.abs(res))
    tol = STAT * (np.abs(yy) + a * np.abs(w) * mag)
    if y is not None:
        assert np.all(np.abs(f64(y) - yy) <= tol + BF16 * np.abs(yy) + 1e-37)
    if r is not None:
        half = 2.0 ** -24 if str(r.dtype).endswith("float32") else BF16
        assert np.all(np.abs(f64(r) - rr) <= STAT * mag + half * np.abs(rr) + 1e-37)
    if quant is not None:
        n, d = yy.shape
        codes, scales = host(quant[0]), f64(quant[1])
        top = np.abs(yy).reshape(n, -1, 128).max(axis=2)
        stol = tol.reshape(n, -1, 128).max(axis=2)
        assert np.all(np.abs(scales - top / 448) <= (stol + STAT * top) / 448 + 1e-37)
        import torch
        val = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
        s8 = np.repeat(scales, 128, axis=1)
        live = s8 > 0
        z = np.where(live, yy / np.where(live, s8, 1.0), 0.0)
        ztol = np.where(live, tol / np.where(live, s8, 1.0), 0.0) + STAT * np.abs(z)
        # the largest value of a group is 448 up to the rounding of its scale
        assert np.all(np.abs(val - z) <= ztol + np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10))
        assert np.all(val[~live] == 0)


CASES = [  # n, d, residual, post, weight, quantize
    (1, 2560, "bf16", False, "bf16", True), (1, 1, "none", False, "f32", False),
    (2, 7, "f32", True, "bf16", False), (5, 64, "bf16", True, "f32", False),
    (63, 128, "none", True, "bf16", True), (64, 2560, "f32", True, "bf16", True),
    (3, 256, "none", False, "f32", True), (300, 777, "bf16", False, "f32", False),
    (2049, 384, "f32", False, "bf16", True), (2050, 512, "none", True, "f32", True),
    (2048, 1000, "bf16", True, "bf16", False), (2047, 1024, "bf16", False, "f32", True),
    (2051, 2048, "f32", True, "f32", True), (2055, 2560, "bf16", True, "bf16", True),
    (130, 1025, "f32", True, "f32", False), (9, 2568, "bf16", True, "bf16", False),
    (17, 4096, "f32", False, "bf16", True), (6, 4097, "bf16", True, "f32", False),
    (5, 8191, "f32", True, "bf16", False), (4, 8192, "bf16", True, "f32", True)]


@pytest.mark.parametrize("n,d,residual,post,weight,quant", CASES)
def test_forward(M, n, d, residual, post, weight, quant):
    say("rms_norm", n, d, residual, post, weight, quant)
    s = make(n * 31 + d, n, d, residual, post, weight)
    y, r, q = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"], quantize=quant)
    assert (r is None) == (residual == "none" and not post)
    check_forward(s, y, r, q)


@pytest.mark.parametrize("n,d,residual,post", [(70, 2560, "bf16", True), (2100, 512, "f32", False),
                                               (33, 8192, "none", True), (2, 24, "bf16", False)])
def test_forward_unaligned_storage(M, n, d, residual, post):
    say("rms_norm, storage off by one element", n, d)
    s = make(n + d, n, d, residual, post, "f32", offset=1)
    y, r, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
    check_forward(s, y, r, None)


@pytest.mark.parametrize("n,d,residual,post,weight,quant", CASES)
def test_backward(M, n, d, residual, post, weight, quant):
    say("rms_norm_backward", n, d, residual, post, weight)
    s = make(n * 37 + d, n, d, residual, post, weight, offset=0 if d % 2 == 0 else 1)
    _, r, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
    r = s["x"] if r is None else r
    dx, dres, dw, dp = M.rms_norm_backward(s["dy"], r, s["w"], EPS, s["dres"],
                                           s["x"] if post else None, s["post"])
    check_backward(s, r, dx, dres, dw, dp)


def check_backward(s, r, dx, dres, dw, dp):
    dy, w, rr = f64(s["dy"]), f64(s["w"]), f64(r)
    dr0 = None if s["dres"] is None else f64(s["dres"])
    post = None if s["post"] is None else f64(s["post"])
    x = f64(s["x"])
    odx, odr, odw, odp = B.rms_norm_backward(dy, rr, w, EPS, dr0, x if post is not None else None, post)
    a = 1 / np.sqrt(np.mean(rr * rr, axis=1, keepdims=True) + EPS)
    nn, h = np.abs(rr * a), np.abs(dy * w)
    mag = a * (h + nn * np.mean(h * nn, axis=1, keepdims=True)) + (0 if dr0 is None else np.abs(dr0))
    half = 2.0 ** -24 if str(dres.dtype).endswith("float32") else BF16
    assert np.all(np.abs(f64(dres) - odr) <= STAT * mag + half * np.abs(odr) + 1e-37)
    assert np.all(np.abs(f64(dw) - odw) <= STAT * np.abs(dy * rr * a).sum(axis=0) + 1e-37)
    if post is None:
        assert np.all(np.abs(f64(dx) - odx) <= STAT * mag + BF16 * np.abs(odx) + 1e-37)
        assert dp is None
        return
    b = 1 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + EPS)
    m, k = np.abs(x * b), mag * np.abs(post)
    size = b * (k + m * np.mean(k * m, axis=1, keepdims=True))
    assert np.all(np.abs(f64(dx) - odx) <= 2 * STAT * size + BF16 * np.abs(odx) + 1e-37)
    assert np.all(np.abs(f64(dp) - odp) <= 2 * STAT * (mag * m).sum(axis=0) + 1e-37)


@pytest.mark.parametrize("n,d,post", [(4099, 2560, True), (5000, 512, False), (3000, 8192, True)])
def test_backward_many_rows_and_repeats(M, n, d, post):
    """More rows than the blocks take at once; the same bits every time."""
    say("rms_norm_backward, many rows", n, d)
    s = make(n, n, d, "f32", post, "bf16")
    _, r, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
    args = (s["dy"], r, s["w"], EPS, s["dres"], s["x"] if post else None, s["post"])
    out = M.rms_norm_backward(*args)
    check_backward(s, r, *out)
    for a, b in zip(out, M.rms_norm_backward(*args)):
        assert (a is None and b is None) or bool((a == b).all())


def test_zero_rows_and_zero_row(M):
    import torch
    say("rms_norm, no rows")
    s = make(1, 0, 256, "bf16", True, "bf16")
    y, r, q = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"], quantize=True)
    assert y.shape == (0, 256) and r.shape == (0, 256) and q[1].shape == (0, 2)
    dx, dres, dw, dp = M.rms_norm_backward(s["dy"], r, s["w"], EPS, s["dres"], s["x"], s["post"])
    assert dx.shape == (0, 256) and float(dw.abs().sum()) == 0.0 and float(dp.abs().sum()) == 0.0
    say("rms_norm, a row of zeros")
    x = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, _, q = M.rms_norm(x, w, EPS, quantize=True)
    assert float(y[0].abs().sum()) == 0.0 and float(q[1][0].abs().sum()) == 0.0
    assert int(q[0][0].sum()) == 0 and float(y[1].float().mean()) == 1.0
    dx, _, _, _ = M.rms_norm_backward(torch.ones_like(x), x, w, EPS)
    # dr = dy / sqrt(eps) at r = 0; at the constant row h - n mean(h n) cancels
    # but for eps: |dx| <= a (1 - a^2) + a few roundings of a
    assert bool((dx[0].float() == torch.tensor(1000.0).bfloat16().item()).all())
    assert float(dx[1].float().abs().max()) < 4e-6


def test_codes_match_the_row_quantiser(M):
    """Where y is exact in bf16, the codes and scales are fp8_quantize_rows'."""
    import torch
    say("rms_norm codes against fp8_quantize_rows")
    # every |x| equal to 2: rms 2, y = x / 2 * w with w a power of two: exact
    sign = torch.randint(0, 2, (70, 512), device="cuda").float() * 2 - 1
    x = (2.0 * sign).bfloat16()
    w = (2.0 ** torch.randint(-6, 7, (512,), device="cuda").float())
    y, _, (codes, scales) = M.rms_norm(x, w, 0.0, quantize=True)
    assert bool((y.float() == sign * w).all())
    c2, s2 = M.fp8_quantize_rows(y)
    assert bool((codes == c2).all()) and bool((scales == s2).all())


def test_inplace_outputs_and_refusals(M):
    import torch
    s = make(5, 40, 384, "f32", True, "bf16")
    say("rms_norm in place")
    y, r, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
    stream = s["res"].clone()
    y2, r2, q = M.rms_norm(s["x"], s["w"], EPS, stream, s["post"], inplace=True, norm_out=False,
                           quantize=True)
    assert r2 is stream and bool((stream == r).all()) and y2 is None and q[0].shape == (40, 384)
    with pytest.raises(ValueError):
        M.rms_norm(s["x"], s["w"], EPS, inplace=True)
    with pytest.raises(ValueError):
        M.rms_norm(s["x"][:, ::2], s["w"][::2], EPS)           # not contiguous
    with pytest.raises(ValueError):
        M.rms_norm(s["x"], s["w"][:383].contiguous(), EPS)
    with pytest.raises(TypeError):
        M.rms_norm(s["x"].float(), s["w"], EPS)
    with pytest.raises(TypeError):
        M.rms_norm(s["x"], s["w"], EPS, post_weight=s["post"].float())
    with pytest.raises(TypeError):
        M.rms_norm(s["x"].cpu(), s["w"], EPS)
    with pytest.raises(M.MoeError):
        M.rms_norm(s["x"][:, :320].contiguous(), s["w"][:320].contiguous(), EPS, quantize=True)
    with pytest.raises(ValueError):
        M.rms_norm_backward(s["dy"], r, s["w"], EPS, x=s["x"])  # x without post_weight


def test_rows_behind_the_batch_stay(M):
    """The C entry writes the n rows it is given and nothing behind them."""
    import torch
    from sigmoid_top_routing_router_amd import _lib
    lib = _lib.load()
    for n, d in ((3, 256), (2049, 256), (5, 77)):
        say("rms_norm, canaries", n, d)
        s = make(n, n, d, "bf16", False, "bf16")
        y = torch.full((n + 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
        r = torch.full((n + 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        _lib.check(lib.moe_rms_norm(s["x"].data_ptr(), s["res"].data_ptr(), None, s["w"].data_ptr(),
                                    n, d, EPS, 0, y.data_ptr(), r.data_ptr(), None, None, st))
        assert bool((y[n:] == 7).all()) and bool((r[n:] == 7).all())
        check_forward(s, y[:n], r[:n], None)


def test_streams_and_graph(M):
    """On a side stream, and captured: every replay gives the eager bits."""
    import torch
    s = make(9, 500, 2560, "bf16", True, "bf16")
    say("rms_norm graph")
    y0, r0, q0 = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"], quantize=True)
    back = M.rms_norm_backward(s["dy"], r0, s["w"], EPS, s["dres"], s["x"], s["post"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, _, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"], stream=side)
    side.synchronize()
    assert bool((y1 == y0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            y, r, q = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"], quantize=True)
            grads = M.rms_norm_backward(s["dy"], r, s["w"], EPS, s["dres"], s["x"], s["post"])
    for rep in range(3):
        for t in (y, r, *grads):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert bool((y == y0).all()) and bool((r == r0).all()) and bool((q[0] == q0[0]).all())
        for a, b in zip(grads, back):
            assert bool((a == b).all()), rep
        M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
        torch.cuda.synchronize()


@pytest.mark.parametrize("n,d", [(4 * 2 ** 20 + 3, 8), (2 ** 20 + 2, 520)])
def test_more_rows_than_one_line_of_blocks(M, n, d):
    """Row n - 1 belongs to a block behind 2^20 others, and its elements lie
    past 2^25 (2^29) of them."""
    import torch
    torch.manual_seed(5)
    x = torch.empty(n, d, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, _ = M.rms_norm(x, w, EPS)[:2]
    for rows in (slice(0, 5), slice(2 ** 20 - 3, 2 ** 20 + 2), slice(n - 5, n)):
        a = f64(x[rows])
        ref = a / np.sqrt((a * a).mean(axis=1, keepdims=True) + EPS)
        assert (np.abs(f64(y[rows]) - ref) <= (STAT + BF16) * np.abs(ref)).all()


def test_nan_rows_show_in_the_codes(M):
    """A NaN in a row makes the row's y NaN; its codes carry it in their scale,
    and the rows beside it stay as they were."""
    import torch
    say("rms_norm, NaN rows")
    s = make(12, 6, 512, "f32", False, "bf16")
    y0, _, (c0, s0) = M.rms_norm(s["x"], s["w"], EPS, s["res"], quantize=True)
    s["res"][2, 300] = float("nan")
    y1, _, (c1, s1) = M.rms_norm(s["x"], s["w"], EPS, s["res"], quantize=True)
    keep = [0, 1, 3, 4, 5]
    assert bool(y1[2].isnan().all()) and bool(s1[2].isnan().all())
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(c0[keep], c1[keep])
    assert torch.equal(s0[keep], s1[keep])

"""rms_norm and rms_norm_backward at the ends of their range: batches without
rows, and rows whose root mean square is far from one."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests.gpu_util import say
from tests.test_gpu_norm import BF16, EPS, STAT, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


@pytest.mark.parametrize("residual", ["none", "bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("weight_grads", [False, True])
def test_backward_of_no_rows(M, residual, post, weight_grads):
    say("rms_norm_backward, no rows", residual, post, weight_grads)
    s = make(1, 0, 256, residual, post, "bf16")
    _, r, _ = M.rms_norm(s["x"], s["w"], EPS, s["res"], s["post"])
    dx, dres, dw, dp = M.rms_norm_backward(s["dy"], s["x"] if r is None else r, s["w"], EPS,
                                           s["dres"], s["x"] if post else None, s["post"],
                                           weight_grads=weight_grads)
    assert dx.shape == dres.shape == (0, 256)
    assert (dw is None) == (not weight_grads) and (dp is None) == (not (weight_grads and post))
    for g in (dw, dp):
        assert g is None or (g.shape == (256,) and not g.any())


def scaled(t, factors):
    """t with its rows times these powers of two (exact)."""
    import torch
    f = torch.from_numpy(factors[:, None]).to(t.device)
    return (t.double() * f).to(t.dtype)


@pytest.mark.parametrize("d,stream,post", [(256, "f32", False), (256, "bf16", True),
                                           (2560, "f32", True), (777, "bf16", False),
                                           (1001, "f32", True)])
def test_rows_far_from_one(M, d, stream, post):
    """eps = 0 and rows from 2^-49 to 2^56 (6e-16 to 7e16), the same batch for r
    and, in the sandwich form, x at scales of its own.  The gradient's terms
    are of order dy / rms, each product of them inside fp32; the bounds are the
    ordinary rows' (relative roundings do not depend on the scale)."""
    say("rms_norm, rows far from one", d, stream, post)
    e = np.array([-49, -45, -43, -42, -30, 0, 0, 30, 42, 45, 47, 50, 56, 0, -49, 47])
    n = len(e)
    s = make(d, n, d, stream, post, "f32")
    s["res"] = scaled(s["res"], 2.0 ** e)
    # the normed x is of order one, x itself only without a second norm
    s["x"] = scaled(s["x"], 2.0 ** (e[::-1] if post else np.minimum(e, 0) - 60))
    y, r, _ = M.rms_norm(s["x"], s["w"], 0.0, s["res"], s["post"])
    x, w, res, dy, dr0 = (f64(s[k]) for k in ("x", "w", "res", "dy", "dres"))
    pw = f64(s["post"]) if post else None
    rr, yy, a = B.rms_norm(x, w, 0.0, res, pw)
    mag = np.abs(rr - res) + np.abs(res)
    assert np.all(np.abs(f64(y) - yy) <= STAT * (np.abs(yy) + a * np.abs(w) * mag)
                  + BF16 * np.abs(yy) + 1e-37)
    half = 2.0 ** -24 if stream == "f32" else BF16
    assert np.all(np.abs(f64(r) - rr) <= STAT * mag + half * np.abs(rr) + 1e-37)

    # backward at rows r of these scales (the sandwich form's sum has its own)
    r = s["res"]
    dx, dres, dw, dp = M.rms_norm_backward(s["dy"], r, s["w"], 0.0, s["dres"],
                                           s["x"] if post else None, s["post"])
    rr = f64(r)
    odx, odr, odw, odp = B.rms_norm_backward(dy, rr, w, 0.0, dr0, x if post else None, pw)
    a = 1 / np.sqrt(np.mean(rr * rr, axis=1, keepdims=True))
    nn, h = np.abs(rr * a), np.abs(dy * w)
    mag = a * (h + nn * np.mean(h * nn, axis=1, keepdims=True)) + np.abs(dr0)
    assert np.all(np.isfinite(f64(dres))) and np.all(np.isfinite(f64(dx)))
    assert np.all(np.abs(f64(dres) - odr) <= STAT * mag + half * np.abs(odr) + 1e-37)
    assert np.all(np.abs(f64(dw) - odw) <= STAT * np.abs(dy * rr * a).sum(axis=0) + 1e-37)
    if not post:
        assert np.all(np.abs(f64(dx) - odx) <= STAT * mag + BF16 * np.abs(odx) + 1e-37)
        return
    b = 1 / np.sqrt(np.mean(x * x, axis=1, keepdims=True))
    m, k = np.abs(x * b), mag * np.abs(pw)
    size = b * (k + m * np.mean(k * m, axis=1, keepdims=True))
    assert np.all(np.abs(f64(dx) - odx) <= 2 * STAT * size + BF16 * np.abs(odx) + 1e-37)
    assert np.all(np.abs(f64(dp) - odp) <= 2 * STAT * (mag * m).sum(axis=0) + 1e-37)

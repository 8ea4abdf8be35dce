"""rms_norm and rms_norm_backward at the ends of their range: batches without
rows."""
import pytest

from tests.gpu_util import say
from tests.test_gpu_norm import EPS, make

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

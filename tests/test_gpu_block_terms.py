"""The block's training step, term by term: what the balance loss and the
load-error injection add to the logits' gradient has to be in it, at its size
and with its sign, and the step's loss, loads and output are right too.

The step's logits, selection and normed rows are taken as they are (they have
tests of their own) and the fp64 forms are evaluated there, so that only the
roundings from there on count.  Tolerances per value: the injection's part as
in its own test (1e-5 of the row's largest), the balance loss's part 3 P of the
size of the terms it is the difference of, P = 2^-18 + max|Z| 2^-22, the
layer's part (C + 2^-18) of its terms with C = (k / 16 + 20) 2^-24, k the
longest sum of the path, and 2^-24 for each of the two additions.  An expert
that a token has not chosen gets nothing from the layer: there the added terms
stand alone."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests import test_gpu_block as block_test
from tests.gpu_util import check_logits, check_output, dev, host, say
from tests.test_gpu_backward import f64
from tests.test_gpu_block import COEF, EPS, LAM, SHAPES, TAU, silu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


@pytest.mark.parametrize("N,d,E,K,h,hs", SHAPES)
def test_added_terms_of_the_step(M, N, d, E, K, h, hs):
    say("block step, terms", N, d, E, K, h, hs)
    P = block_test.block(N + d, N, d, E, K, h, hs)
    T, W = block_test.to_dev(M, P)
    cuts = [0, N // 3, N // 3, N - 5, N]
    got = block_test.step(M, T, W, K, dev(np.array(cuts, np.int32)))
    spans = list(zip(cuts[:-1], cuts[1:]))
    y = f64(M.rms_norm(T["sub"], T["w"], EPS, T["stream"], T["post"])[0])
    f = {k: (O.bf16_to_f32(v) if v.dtype == np.uint16 else v).astype(np.float64)
         for k, v in P.items()}
    Z, ids = host(got["Z"]), host(got["ids"])
    check_logits(Z, y @ f["w_router"].T)

    # the loss and its loads
    counts = B.segment_counts(ids, E, spans)
    share = 2.0 ** -18 + float(np.abs(Z).max()) * 2.0 ** -22
    loss = B.balance_loss(Z, counts, COEF, "sigmoid_norm", spans)[0]
    assert loss > 0 and abs(float(got["loss"][0]) - loss) <= share * loss

    # the layer's output
    shared = (f["ws_gate"][0], f["ws_up"][0], f["ws_down"][0]) if hs else None
    out = np.zeros((N, d))
    for e in range(E):
        t, k = np.nonzero(ids == e)
        if len(t):
            H = silu(y[t] @ f["w_gate"][e].T) * (y[t] @ f["w_up"][e].T)
            s = 1.0 / (1.0 + np.exp(-Z[t, e].astype(np.float64)))
            np.add.at(out, t, s[:, None] * (H @ f["w_down"][e].T))
    if hs:
        out += (silu(y @ shared[0].T) * (y @ shared[1].T)) @ shared[2].T
    check_output(f64(got["out"]), out, "step output")

    # the logits' gradient and its three terms
    lei = O.lei_backward(Z, ids, None, LAM, TAU)[1]
    balance, size = B.balance_loss_backward(Z, counts, COEF, "sigmoid_norm", spans)
    want, mag = B.layer_backward(y, f["dy"], Z, ids, f["w_router"], f["w_gate"], f["w_up"],
                                 f["w_down"], shared, lei + balance)
    want, mag = want["logits"], mag["logits"]
    c = (max(N, d, h, E, hs) / 16 + 20) * 2.0 ** -24
    tol = 1e-5 * np.abs(lei).max(axis=1, keepdims=True) + 3 * share * size
    tol = tol + (c + 2.0 ** -18) * mag + 2.0 ** -24 * (np.abs(lei + balance) + np.abs(want)) + 1e-37
    dz = f64(got["logits"])
    assert np.all(np.abs(dz - want) <= tol)

    # a term that is lost, doubled or turned round leaves these bounds nearly
    # everywhere that the layer itself adds nothing
    alone = np.ones((N, E), bool)
    alone[np.arange(N)[:, None], ids] = False
    for name, term in (("injection", lei), ("balance loss", balance)):
        for factor in (-1.0, 1.0, -2.0):
            seen = np.abs(dz - (want + factor * term)) > tol
            say(name, factor, f"{seen[alone].mean():.3f}")
            assert seen[alone].mean() > 0.9, (name, factor)

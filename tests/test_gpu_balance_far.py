"""The balance loss of rows whose logits are all far below zero: every sigma of
such a row is below fp32's (fp64's) smallest number, their ratios are not.
Tolerances as in test_gpu_balance, by the largest |logit|."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests.gpu_util import dev, host, say
from tests.test_gpu_balance import SCORES, bounds, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def far_rows(N, E, seed):
    """Rows around 0, -30, -86, -90, -103, -200 and -1000 in turn, and a row of
    each kind that one expert leaves."""
    rng = np.random.default_rng(seed)
    at = np.array([0, -30, -86, -90, -103, -200, -1000], np.float32)
    Z = (at[np.arange(N) % 7][:, None] + rng.standard_normal((N, E))).astype(np.float32)
    Z[7:14, E // 2] = [3.0, -1.0, -85.0, -2.0, 60.0, -150.0, 0.0]
    return Z, np.argsort(-Z, axis=1)[:, :2].astype(np.int32)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N,E", [(35, 33), (700, 384), (64, 100)])
def test_rows_far_below_zero(M, score, N, E):
    say("balance, rows far below zero", score, N, E)
    Z, ids = far_rows(N, E, N)
    check(M, Z, ids, [(0, N // 3), (N // 3, N)], score)
    for lo in (3, 4, 5, 6):                               # such rows alone in a segment
        if score != "sigmoid":
            check(M, Z, ids, [(lo, lo + 1)], score)
            continue
        # its scores themselves are subnormal: one below 2^-126 counts as 0, and
        # so the loss, coef sum f P with sum f = E, is off by coef E 2^-126 at most
        counts = B.segment_counts(ids, E, [(lo, lo + 1)])
        want, omean = B.balance_loss(Z, counts, 0.02, score, [(lo, lo + 1)])
        loss, _, mean = M.balance_loss(dev(Z), dev(ids), 0.02, score, bounds([(lo, lo + 1)]))
        tol = 2.0 ** -18 + 1010 * 2.0 ** -22
        assert abs(float(loss[0]) - want) <= tol * want + 0.02 * E * 2.0 ** -126
        assert np.all(np.abs(host(mean) - omean) <= tol * omean + 2.0 ** -126)


def test_the_lowest_value(M):
    """All logits of a row at fp32's lowest, or at -1e30: the scores are equal."""
    say("balance, the lowest value")
    E = 40
    Z = np.full((6, E), np.finfo(np.float32).min, np.float32)
    Z[3:] = -1e30
    ids = np.tile(np.array([[0, 1]], np.int32), (6, 1))
    for score in ("sigmoid_norm", "softmax"):
        loss, counts, mean = M.balance_loss(dev(Z), dev(ids), 0.02, score)
        assert np.all(np.abs(host(mean) - 1 / E) <= 2.0 ** -18 / E)
        assert abs(float(loss[0]) - 0.02) <= 2.0 ** -18 * 0.02   # f sums to E, P is 1 / E
        dz = host(M.balance_loss_backward(dev(Z), counts, 0.02, score)).astype(np.float64)
        # p (f - 1) coef / T, sigma(-z) being 1
        f = np.zeros(E)
        f[:2] = E / 2
        want = 0.02 / 6 / E * (f - 1.0)
        assert np.all(np.abs(dz - want) <= 3 * 2.0 ** -18 * 0.02 / 6 / E * (f + 1.0))


@pytest.mark.parametrize("score", ["sigmoid_norm", "softmax"])
def test_masked_experts(M, score):
    """Experts at -inf have the score 0 and no gradient; the others are the rows
    without them.  A row with all of them there has no score: NaN."""
    say("balance, masked experts", score)
    rng = np.random.default_rng(4)
    E, keep = 50, np.arange(0, 50, 3)
    Z = (rng.standard_normal((20, E)) - 95).astype(np.float32)
    small, ids = np.ascontiguousarray(Z[:, keep]), np.zeros((20, 1), np.int32)
    Z[:, np.setdiff1d(np.arange(E), keep)] = -np.inf
    counts = B.segment_counts(ids, E, [(0, 20)])
    loss, c, mean = M.balance_loss(dev(Z), dev(ids), 0.02, score)
    _, omean = B.balance_loss(small, counts[:, keep], 0.02, score, [(0, 20)])
    tol = 2.0 ** -18 + 100 * 2.0 ** -22
    got = host(mean)
    assert np.all(np.abs(got[:, keep] - omean) <= tol * omean)
    assert got.sum() == got[:, keep].sum()
    odz, size = B.balance_loss_backward(small, counts[:, keep] * len(keep), 0.02, score, [(0, 20)])
    dz = host(M.balance_loss_backward(dev(Z), c, 0.02, score)).astype(np.float64)
    # f = E on expert 0: E / len(keep) times what it is over the kept ones
    scale = E / len(keep)
    assert np.all(np.abs(dz[:, keep] - scale * odz) <= 3 * tol * scale * size + 1e-37)
    assert not dz[:, np.setdiff1d(np.arange(E), keep)].any()
    Z[7] = -np.inf
    seg = bounds([(0, 7), (7, 8), (8, 20)])
    loss, c, mean = M.balance_loss(dev(Z), dev(ids), 0.02, score, seg)
    got = host(mean)
    assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2]]).all() and np.isnan(float(loss[0]))

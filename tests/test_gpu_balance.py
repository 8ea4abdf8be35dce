"""GPU parity of moe_balance_loss and moe_balance_loss_backward against the
plain fp64 forms.

Tolerances, with Z the largest |logit| of the batch: exp(-|z|) through a base-2
exponential rounds its argument (|z| 2^-24 relative, twice that for z - max)
and its result (2^-23), a reciprocal and the sums over a row (24 values of a
lane, four steps) and over a block's rows (at most 16 rows of a lane, six
steps) add below 2^-19 together.  A score, and a mean of scores, is therefore
off by at most P = 2^-18 + Z 2^-22 relative, a gradient by 3 P of the size of
the terms that it is the difference of.  Loads are equal."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from synth import make_bias, make_logits
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu

SCORES = ["sigmoid", "sigmoid_norm", "softmax"]


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def spans_of(kind, N, rng):
    """Segments of a batch of N rows: (begin, end) pairs."""
    if kind == "one":
        return [(0, N)]
    if kind == "rows":
        return [(t, t + 1) for t in range(N)]
    if kind == "empty":
        return [(0, 0)] * 3
    if kind == "inside":
        return [(N // 3, N // 3), (N // 3, (2 * N) // 3), (N - 1, N - 1)]
    cut = np.sort(rng.integers(0, N + 1, kind - 1))
    edge = np.concatenate([[0], cut, [N]])
    out = []
    for lo, hi in zip(edge[:-1], edge[1:]):
        out.append((int(lo), int(hi - rng.integers(0, (hi - lo) // 8 + 1))))
    return out


def make(seed, N, E, K, std=2.0):
    Z = make_logits(seed, N, E, std)
    off = np.linspace(1.0, -1.0, E).astype(np.float32)
    ids, _, _ = O.route((Z + off).astype(np.float32), make_bias(seed + 1, E, 0.1), K)
    return Z, ids.astype(np.int32)


def bounds(spans):
    return (dev(np.array([s[0] for s in spans], np.int32)),
            dev(np.array([s[1] for s in spans], np.int32)))


def check(M, Z, ids, spans, score, coef=0.02, segments="pairs", grad=None, grad_loss=None,
          counts=None, inplace=False):
    N, E = Z.shape
    seg = None if segments is None else bounds(spans)
    Zd = dev(Z)
    loss, cnt, mean = M.balance_loss(Zd, dev(ids), coef, score, seg,
                                     counts=None if counts is None else dev(counts))
    own = B.segment_counts(ids, E, spans)
    assert np.array_equal(host(cnt), own)
    used = own if counts is None else counts.astype(np.int64)
    inside = np.zeros(N, bool)
    for lo, hi in spans:
        inside[lo:hi] = True
    zmax = float(np.abs(Z[inside]).max()) if inside.any() else 0.0
    tol = 2.0 ** -18 + zmax * 2.0 ** -22
    oloss, omean = B.balance_loss(Z, used, coef, score, spans)
    assert np.all(np.abs(host(mean) - omean) <= tol * omean + 1e-37)
    assert abs(float(loss[0]) - oloss) <= tol * abs(oloss)
    odz, size = B.balance_loss_backward(Z, used, coef, score, spans)
    gl = 1.0 if grad_loss is None else grad_loss
    gd = None if grad is None else dev(grad)
    dz = M.balance_loss_backward(Zd, cnt if counts is None else dev(counts), coef, score, seg,
                                 None if grad_loss is None else dev(np.array([gl], np.float32)),
                                 gd, inplace=inplace)
    assert (dz is gd) == inplace
    base = 0.0 if grad is None else grad.astype(np.float64)
    want = base + gl * odz
    got = host(dz).astype(np.float64)
    assert np.all(np.abs(got - want) <= 3 * tol * abs(gl) * size + 2.0 ** -24 * np.abs(want) + 1e-37)
    assert np.array_equal(got[~inside], np.broadcast_to(base, got.shape)[~inside])
    return loss, cnt, mean, dz


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N,E,K,kind", [
    (1, 9, 8, "one"), (1, 2, 1, "one"), (15, 64, 3, "one"), (16, 65, 4, "inside"),
    (333, 100, 5, 9), (64, 384, 6, "rows"), (1000, 384, 6, "one"), (1025, 128, 8, 17),
    (257, 383, 7, "empty"), (2000, 20, 4, 64)])
def test_parity(M, score, N, E, K, kind):
    say("balance", score, N, E, K, kind)
    rng = np.random.default_rng(N + E)
    Z, ids = make(600 + N, N, E, K)
    check(M, Z, ids, spans_of(kind, N, rng), score)


@pytest.mark.parametrize("score,N,kind", [("sigmoid_norm", 16384, 7), ("softmax", 5003, "rows"),
                                          ("sigmoid", 40000, "one")])
def test_parity_large(M, score, N, kind):
    """More rows than one block takes, segments that cross blocks, and a segment
    for every row; with an added gradient."""
    say("balance large", score, N, kind)
    rng = np.random.default_rng(N)
    Z, ids = make(700 + N, N, 384, 6)
    grad = (rng.standard_normal(Z.shape) * 1e-6).astype(np.float32)
    check(M, Z, ids, spans_of(kind, N, rng), score, grad=grad, grad_loss=0.75)


@pytest.mark.parametrize("score", SCORES)
def test_no_segments_argument_offsets_and_inplace(M, score):
    import torch
    Z, ids = make(41, 500, 96, 3)
    say("balance without segments", score)
    grad = (np.random.default_rng(3).standard_normal(Z.shape) * 1e-4).astype(np.float32)
    check(M, Z, ids, [(0, 500)], score, segments=None, grad=grad, grad_loss=-2.0, inplace=True)
    say("balance with offsets", score)
    cu = np.array([0, 17, 17, 300, 500], np.int32)
    a = M.balance_loss(dev(Z), dev(ids), 0.02, score, dev(cu))
    b = M.balance_loss(dev(Z), dev(ids), 0.02, score, (dev(cu[:-1]), dev(cu[1:])))
    for x, y in zip(a, b):
        assert bool((x == y).all())
    assert torch.equal(M.balance_loss_backward(dev(Z), a[1], 0.02, score, dev(cu)),
                       M.balance_loss_backward(dev(Z), a[1], 0.02, score,
                                               (dev(cu[:-1]), dev(cu[1:]))))


@pytest.mark.parametrize("score", SCORES)
def test_given_counts_and_missing_ids(M, score):
    """Loads of the whole job in place of the batch's own; ids outside [0, E) are
    not counted; a segment without any load contributes nothing."""
    Z, ids = make(42, 300, 50, 4)
    ids[::3] = -1
    ids[100:200] = 50 + ids[100:200]                          # its -1 become 49
    spans = [(0, 100), (100, 200), (210, 300)]
    say("balance, ids outside the range", score)
    check(M, Z, ids, spans, score)
    ids[100:200:3], ids[101:200:3], ids[102:200:3] = -5, 50, 1 << 30
    own = B.segment_counts(ids, 50, spans)
    assert own[1].sum() == 0                                  # no load in segment 1
    check(M, Z, ids, spans, score)
    say("balance, given counts", score)
    counts = np.random.default_rng(5).integers(0, 1 << 30, own.shape).astype(np.int32)
    check(M, Z, ids, spans, score, counts=counts)
    loss, cnt, _ = M.balance_loss(dev(Z), None, 0.02, score, bounds(spans), counts=dev(counts))
    want, _ = B.balance_loss(Z, counts.astype(np.int64), 0.02, score, spans)
    assert abs(float(loss[0]) - want) <= 2.0 ** -17 * abs(want)
    assert np.array_equal(host(cnt), counts)


@pytest.mark.parametrize("score", SCORES)
def test_rows_outside_hold_anything(M, score):
    """NaN and infinities in rows of no segment reach nothing."""
    Z, ids = make(43, 400, 72, 4)
    spans = [(10, 130), (130, 130), (140, 390)]
    say("balance, rows outside", score)
    ref = check(M, Z, ids, spans, score)
    bad = Z.copy()
    bad[:10], bad[130:140], bad[390:] = np.nan, np.inf, -np.inf
    ids2 = ids.copy()
    ids2[:10], ids2[390:] = 0, 71
    loss, cnt, mean = M.balance_loss(dev(bad), dev(ids2), 0.02, score, bounds(spans))
    dz = M.balance_loss_backward(dev(bad), cnt, 0.02, score, bounds(spans))
    for a, b in zip(ref, (loss, cnt, mean, dz)):
        assert np.array_equal(host(a), host(b))
    assert not host(dz)[:10].any()


@pytest.mark.parametrize("score", SCORES)
def test_far_logits(M, score):
    """Logits up to 80 from zero, of both signs and all equal."""
    rng = np.random.default_rng(8)
    Z = rng.uniform(-80, 80, (50, 33)).astype(np.float32)
    Z[3], Z[4], Z[5] = 80.0, -80.0, 0.0
    ids = np.argsort(-Z, axis=1)[:, :3].astype(np.int32)
    say("balance, far logits", score)
    check(M, Z, ids, [(0, 50)], score)


@pytest.mark.parametrize("E", [96, 97])
def test_unaligned_storage(M, E):
    import torch
    Z, ids = make(44, 200, E, 3)
    say("balance, storage off by one element", E)
    flat = torch.empty(Z.size + 1, device="cuda")
    flat[1:] = dev(Z).view(-1)
    view = flat[1:].view(200, E)
    a = M.balance_loss(view, dev(ids), 0.02, "softmax")
    b = M.balance_loss(dev(Z), dev(ids), 0.02, "softmax")
    for x, y in zip(a, b):
        assert bool((x == y).all())
    assert torch.equal(M.balance_loss_backward(view, a[1], 0.02, "softmax"),
                       M.balance_loss_backward(dev(Z), a[1], 0.02, "softmax"))


def test_segments_that_are_not_ascending_stay_inside(M):
    """Unspecified values, but no access out of range and no hang."""
    Z, ids = make(45, 200, 40, 3)
    say("balance, bad segments")
    b = dev(np.array([500, -7, 150, 20], np.int32))
    e = dev(np.array([900, 1 << 30, 10, 180], np.int32))
    loss, cnt, mean = M.balance_loss(dev(Z), dev(ids), 0.02, "sigmoid", (b, e))
    dz = M.balance_loss_backward(dev(Z), cnt, 0.02, "sigmoid", (b, e))
    assert host(dz).shape == (200, 40) and host(cnt).shape == (4, 40)


def test_repeats_streams_and_graph(M):
    import torch
    Z, ids = make(46, 3000, 384, 6)
    spans = spans_of(12, 3000, np.random.default_rng(1))
    seg, Zd, idd = bounds(spans), dev(Z), dev(ids)
    say("balance graph")

    def run(stream=None):
        loss, cnt, mean = M.balance_loss(Zd, idd, 0.02, "sigmoid_norm", seg, stream=stream)
        return loss, cnt, mean, M.balance_loss_backward(Zd, cnt, 0.02, "sigmoid_norm", seg,
                                                        stream=stream)
    ref = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = run(side)
    side.synchronize()
    for a, b in zip(ref, out):
        assert bool((a == b).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            cap = run()
    for rep in range(3):
        for t in cap:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, cap):
            assert bool((a == b).all()), rep
        run()
        torch.cuda.synchronize()


def test_refusals(M):
    Z, ids = make(47, 20, 12, 3)
    Zd, idd = dev(Z), dev(ids)
    say("balance refusals")
    cu = dev(np.array([0, 20], np.int32))
    cnt = M.balance_loss(Zd, idd)[1]
    for bad in (lambda: M.balance_loss(Zd), lambda: M.balance_loss(Zd, idd, score="tanh"),
                lambda: M.balance_loss(Zd, idd[:10].contiguous()),
                lambda: M.balance_loss(Zd, idd, segments=cu[:1].contiguous()),
                lambda: M.balance_loss(Zd, idd, counts=cnt[:, :5].contiguous()),
                lambda: M.balance_loss_backward(Zd, None),
                lambda: M.balance_loss_backward(Zd, cnt, inplace=True),
                lambda: M.balance_loss_backward(Zd, cnt, grad_loss=Zd[0].contiguous())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: M.balance_loss(Zd.double(), idd), lambda: M.balance_loss(Zd, idd.long()),
                lambda: M.balance_loss(Zd, idd, segments=cu.long()),
                lambda: M.balance_loss(Zd, idd.cpu())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(M.MoeError):
        M.balance_loss(Zd, idd, coef=float("nan"))

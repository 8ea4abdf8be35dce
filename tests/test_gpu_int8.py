"""GPU parity of the 8-bit integer operators against the fp64 forms.

Tolerances.  The integers and the sums of their products are exact.  U = 2^-24:
the sum's conversion, the product of the scales and its product with the sum
round once each, 3 U; bf16 adds HALF = 2^-8.  silu(g) u: exp of -g is that of a
product rounded once (|g| 2 U relative) in the hardware's own 2^-21, its sum,
the reciprocal (2^-22) and three products: |g| 2^-22 + 2^-19 with the operands'
own 3 U (which silu enlarges by at most 1 + |g|)."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu

U, HALF, TINY = 2.0 ** -24, 2.0 ** -8, 1e-35


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


def bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


@pytest.mark.parametrize("n,cols", [(1, 16), (3, 48), (64, 2560), (1, 65536), (130, 8192),
                                    (257, 8208), (5, 512), (1000, 1040), (7, 1024), (9, 3056),
                                    (6, 3088), (3, 16384), (3, 16400)])
def test_quantize_rows(M, n, cols):
    say("quantize", n, cols)
    rng = np.random.default_rng(n + cols)
    x = rng.standard_normal((n, cols)) * np.exp2(rng.integers(-30, 30, (n, 1)))
    x[:, 3] *= 30
    if n > 2:
        x[0] = 0
        x[1] = 0
        x[1, cols - 1] = -1.0          # one value, the last
        x[2, 1:9] = x[2].max() / 2     # halves of the largest
    t = bf16(x)
    codes, scales = M.int8_quantize_rows(t)
    q, s = R.int8_quantize(f64(t))
    assert np.array_equal(host(codes), q)
    assert np.array_equal(host(scales), s)


def test_quantize_every_significand(M):
    """Every significand of the largest value against every smaller value, at a
    large, a middle and a tiny exponent (where s is subnormal), and the largest."""
    sig = np.arange(128, 256) / 128.0
    for e in (-130, -118, -60, -59, 0, 127):
        x = np.zeros((128, 2048))
        x[:, 0] = sig
        small = (np.arange(128, 256)[None, :] / 128.0 * np.exp2(-np.arange(1, 11))[:, None]).reshape(-1)
        x[:, 1:1281] = -small
        t = bf16(np.ldexp(x, e))
        codes, scales = M.int8_quantize_rows(t)
        q, s = R.int8_quantize(f64(t))
        assert np.array_equal(host(scales), s), e
        assert np.array_equal(host(codes), q), e


def test_quantize_not_finite(M):
    x = np.ones((5, 64))
    t = bf16(x)
    t[1, 7] = float("nan")
    t[2, 63] = float("inf")
    t[3, 0] = float("-inf")
    codes, scales = M.int8_quantize_rows(t)
    s, c = host(scales), host(codes)
    assert np.all(np.isnan(s[1:4])) and np.all(np.isfinite(s[[0, 4]]))
    assert np.all(c[1:4] == 0) and np.all(c[[0, 4]] == 127)
    # what is multiplied with such a row is NaN, its neighbours are not
    w = M.int8_quantize_rows(bf16(np.ones((24, 64))))
    y = f64(M.int8_matmul((codes, scales), w))
    assert np.all(np.isnan(y[1:4])) and np.all(y[[0, 4]] == 64)


def integers(rng, shape, extreme=False):
    import torch
    if extreme:
        a = np.full(shape, -128)
    else:
        a = rng.integers(-128, 128, shape)
    return torch.from_numpy(a.astype(np.int8)).cuda()


def scales(rng, shape, std=1.0):
    import torch
    return torch.from_numpy((std * (0.5 + rng.random(shape))).astype(np.float32)).cuda()


def check(y, q, s, w, w_up):
    """Rows y of one weight."""
    g = R.int8_product(host(q), host(s), host(w[0]), host(w[1]))
    if w_up is None:
        assert np.all(np.abs(y - g) <= (3.1 * U + HALF) * np.abs(g) + TINY)
        return
    u = R.int8_product(host(q), host(s), host(w_up[0]), host(w_up[1]))
    h = R.silu(g) * u
    tol = (HALF + 2.0 ** -19 + np.abs(g) * 2.0 ** -22) * np.abs(h) + TINY * (1 + np.abs(u))
    assert np.all(np.abs(y - h) <= tol)


DENSE = [  # n, k, cols
    (1, 16, 8), (1, 2560, 512), (1, 48, 24), (7, 144, 40), (16, 256, 256), (17, 272, 264),
    (33, 1024, 96), (64, 512, 2560), (65, 4112, 136), (128, 128, 128), (129, 400, 520),
    (255, 160, 1000), (257, 656, 264), (300, 2560, 384), (513, 80, 72), (1000, 512, 8),
    (2, 65536, 16), (40, 16, 4096),
]


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("n,k,cols", DENSE)
def test_dense(M, n, k, cols, up):
    say("dense", n, k, cols, up)
    rng = np.random.default_rng(n * 7 + k + cols)
    q, s = integers(rng, (n, k)), scales(rng, n, 1 / np.sqrt(k) / 5000)
    w = integers(rng, (cols, k)), scales(rng, cols)
    w_up = (integers(rng, (cols, k)), scales(rng, cols)) if up else None
    check(f64(M.int8_matmul((q, s), w, w_up=w_up)), q, s, w, w_up)


def test_largest_sums(M):
    """-128 times -128 over the longest k: 2^30, and a silu far from zero on both
    sides."""
    rng = np.random.default_rng(1)
    q, s = integers(rng, (3, 65536), True), scales(rng, 3, 2.0 ** -26)
    w = integers(rng, (8, 65536), True), scales(rng, 8)
    check(f64(M.int8_matmul((q, s), w)), q, s, w, None)
    up = integers(rng, (8, 65536)), scales(rng, 8)
    w[1][:4] *= 40
    w[0][4:] = 127
    w[1][4:] *= 40
    check(f64(M.int8_matmul((q, s), w, w_up=up)), q, s, w, up)


GROUPED = [  # N, E, K, k, cols, share: how the pairs fall
    (1, 384, 6, 2560, 64, "even"), (1, 3, 1, 16, 8, "even"), (64, 20, 6, 512, 136, "even"),
    (64, 384, 6, 128, 32, "even"), (300, 4, 2, 272, 264, "away"), (700, 3, 2, 160, 72, "one"),
    (90, 7, 8, 400, 520, "away"), (37, 5, 3, 1040, 256, "all"), (1500, 4, 4, 64, 96, "even"),
    (515, 2, 1, 96, 300 * 8, "even"), (2000, 6, 1, 48, 16, "steps"),
]


def pairs(rng, N, E, K, share):
    import torch
    if share == "away":
        ids = rng.integers(-2, E + 2, (N, K))
    elif share == "one":
        ids = np.full((N, K), E - 1)
    elif share == "all":
        ids = np.full((N, K), -1)
    elif share == "steps":  # loads of 1, 63, 64, 65, 255, ...
        ids = np.searchsorted(np.cumsum([1, 63, 257, 289, 256]), np.arange(N), side="right")[:, None]
        ids = np.repeat(ids, K, 1)
    else:
        ids = np.argsort(rng.random((N, max(E, K))), axis=1)[:, :K] % E
    return torch.from_numpy(ids.astype(np.int32)).cuda()


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,E,K,k,cols,share", GROUPED)
def test_grouped(M, N, E, K, k, cols, share, gather, up):
    import torch
    say("grouped", N, E, K, k, cols, share, gather, up)
    rng = np.random.default_rng(N + E + k)
    ids = pairs(rng, N, E, K, share)
    g = M.group_tokens(ids, E)
    n = N if gather else N * K
    q, s = integers(rng, (n, k)), scales(rng, n, 1 / np.sqrt(k) / 5000)
    w = integers(rng, (E, cols, k)), scales(rng, (E, cols))
    w_up = (integers(rng, (E, cols, k)), scales(rng, (E, cols))) if up else None
    out = torch.full((N * K, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    y = f64(M.int8_matmul((q, s), w, w_up=w_up, grouping=g, gather=gather, out=out))
    offsets, src = host(g.offsets), host(g.sorted_src)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi == lo:
            continue
        rows = torch.from_numpy(src[lo:hi] // K if gather else np.arange(lo, hi)).long().cuda()
        check(y[lo:hi], q[rows], s[rows], (w[0][e], w[1][e]),
              None if w_up is None else (w_up[0][e], w_up[1][e]))
    assert np.all(y[offsets[-1]:] == 7.0)


def test_offsets_that_do_not_ascend_stay_in_range(M):
    """Unspecified rows, but nothing outside of out is touched."""
    import torch
    rng = np.random.default_rng(2)
    rows, k, cols, E = 200, 64, 40, 5
    q, s = integers(rng, (rows, k)), scales(rng, rows)
    w = integers(rng, (E, cols, k)), scales(rng, (E, cols))
    pos = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    for offs in ([0, 200, 0, 200, 0, 200], [-5, 1 << 30, -(1 << 31), 300, 100, 50],
                 [200, 200, 200, 200, 200, 200]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        guard = torch.full((rows + 64, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        src = torch.tensor(rng.integers(-2 ** 31, 2 ** 31, rows), dtype=torch.int64).int().cuda()
        g = M.Grouping(None, off, src, pos)
        for gather in (False, True):
            M.int8_matmul((q, s), w, grouping=g, gather=gather, out=guard[32:32 + rows])
        torch.cuda.synchronize()
        assert bool((guard[:32] == 7).all()) and bool((guard[32 + rows:] == 7).all())
        if offs[0] == 200:
            assert bool((guard == 7).all())


def test_rows_and_weights_past_four_gigabytes(M):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    # a of 4.6 GB; the last rows are checked
    n, k, cols = 70000, 65536, 8
    q = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    tail = torch.randint(-128, 128, (300, k), generator=gen, device="cuda").to(torch.int8)
    q[-300:] = tail
    s = torch.rand(n, generator=gen, device="cuda")
    w = (torch.randint(-128, 128, (cols, k), generator=gen, device="cuda").to(torch.int8),
         torch.rand(cols, generator=gen, device="cuda"))
    y = M.int8_matmul((q, s), w)
    check(f64(y[-300:]), tail, s[-300:], w, None)
    assert bool((y[:-300] == 0).all())
    del q, y
    # weights of 5.4 GB, the last experts used; out of 4.3 GB
    E, cols, k, N = 80, 65536, 1024, 33000
    wq = torch.zeros(E, cols, k, dtype=torch.int8, device="cuda")
    wq[-1] = torch.randint(-128, 128, (cols, k), generator=gen, device="cuda").to(torch.int8)
    ws = torch.rand(E, cols, generator=gen, device="cuda")
    ids = torch.full((N, 1), E - 1, dtype=torch.int32, device="cuda")
    g = M.group_tokens(ids, E)
    q = torch.randint(-128, 128, (N, k), generator=gen, device="cuda").to(torch.int8)
    s = torch.rand(N, generator=gen, device="cuda")
    y = M.int8_matmul((q, s), (wq, ws), grouping=g)
    c = slice(cols - 64, cols)
    for rows in (slice(0, 40), slice(N - 40, N)):
        check(f64(y[rows, c]), q[rows], s[rows], (wq[-1][c], ws[-1][c]), None)


def test_repeatable_streams_and_graphs(M):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    N, E, K, k, cols = 500, 8, 2, 512, 320
    ids = torch.randint(-1, E, (N, K), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.randn(N, k, generator=gen, device="cuda").bfloat16()
    w = M.int8_quantize_rows(torch.randn(E, cols, k, generator=gen, device="cuda").bfloat16())
    u = M.int8_quantize_rows(torch.randn(E, cols, k, generator=gen, device="cuda").bfloat16())
    assert w[0].shape == (E, cols, k) and w[1].shape == (E, cols)
    out = torch.zeros(N * K, cols, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        g = M.group_tokens(ids, E, stream=stream)
        q = M.int8_quantize_rows(x, stream=stream)
        return M.int8_matmul(q, w, w_up=u, grouping=g, gather=True, out=out, stream=stream)
    want = call().clone()
    assert torch.equal(call(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        x.copy_(torch.randn(N, k, generator=gen, device="cuda").bfloat16())
        ids.copy_(torch.randint(-1, E, (N, K), generator=gen, device="cuda", dtype=torch.int32))
        out.zero_()
        eager = call().clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_refusals(M):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q = M.int8_quantize_rows(x)
    w = M.int8_quantize_rows(torch.zeros(24, 64, dtype=torch.bfloat16, device="cuda"))
    we = M.int8_quantize_rows(torch.zeros(3, 24, 64, dtype=torch.bfloat16, device="cuda"))
    g = M.group_tokens(torch.zeros(2, 2, dtype=torch.int32, device="cuda"), 3)
    bad = [
        (TypeError, lambda: M.int8_quantize_rows(x.float())),
        (ValueError, lambda: M.int8_quantize_rows(x[0])),
        (M.MoeError, lambda: M.int8_quantize_rows(x[:, :24].contiguous())),
        (TypeError, lambda: M.int8_matmul((q[0].view(torch.uint8), q[1]), w)),
        (ValueError, lambda: M.int8_matmul((q[0], None), w)),
        (ValueError, lambda: M.int8_matmul((q[0], q[1][:3]), w)),
        (ValueError, lambda: M.int8_matmul(q, (w[0], None))),
        (ValueError, lambda: M.int8_matmul(q, (w[0][:, :48].contiguous(), w[1]))),
        (ValueError, lambda: M.int8_matmul(q, we)),
        (ValueError, lambda: M.int8_matmul(q, w, grouping=g)),
        (ValueError, lambda: M.int8_matmul(q, w, gather=True)),
        (ValueError, lambda: M.int8_matmul(q, we, grouping=g, gather=True)),
        (ValueError, lambda: M.int8_matmul((q[0][:3], q[1][:3]), we, grouping=g)),
        (ValueError, lambda: M.int8_matmul(q, w, w_up=(w[0][:8], w[1][:8]))),
        (ValueError, lambda: M.int8_matmul(q, w, out=x)),
        (M.MoeError, lambda: M.int8_matmul(q, (w[0][:20], w[1][:20]))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert M.int8_matmul((q[0][:0], q[1][:0]), w).shape == (0, 24)


# Shapes large enough for the tiles of 64, 128, 192 and 256 rows, one to six stages
# deep, and for the few-row forms that the lists above do not reach.
DENSE_LARGE = [  # n, k, cols
    (34, 48, 4112), (38, 384, 2272), (288, 32, 264), (35, 272, 4072),
    (130, 48, 4024), (147, 160, 4160), (133, 320, 4136),
    (5661, 16, 528), (5969, 144, 520), (5751, 272, 520), (5910, 16, 296), (5616, 400, 280),
    (4695, 16, 1568), (4127, 144, 1800), (5457, 272, 1296), (5420, 16, 664), (4652, 656, 776),
    (5489, 16, 2064), (4419, 144, 2600), (4821, 656, 2312), (1354, 16, 4128), (1731, 144, 3224),
]
GROUPED_LARGE = [  # N, E, K, k, cols
    (5, 8, 1, 176, 3160), (101, 8, 3, 336, 3176), (8, 8, 1, 144, 640), (57, 3, 1, 288, 2032),
    (5303, 5, 1, 16, 528), (5381, 5, 1, 272, 536), (2783, 5, 2, 144, 528), (330, 8, 1, 16, 3792),
    (101, 8, 3, 656, 3848), (1541, 8, 1, 16, 4128), (786, 8, 2, 272, 3904), (577, 8, 1, 16, 3952),
    (188, 8, 3, 400, 3928), (2365, 8, 1, 16, 3856), (1263, 8, 2, 656, 3728), (266, 8, 3, 144, 4088),
]


def check_large(y, q, s, w, w_up):
    """check with the product by torch in 64 bits (sums below 2^53: exact)."""
    def product(v):
        return (q.double() @ v[0].double().T) * s.double()[:, None] * v[1].double()[None, :]
    g, y = product(w), y.double()
    if w_up is None:
        assert bool(((y - g).abs() <= (3.1 * U + HALF) * g.abs() + TINY).all())
        return
    u = product(w_up)
    h = g / (1 + (-g).exp()) * u
    tol = (HALF + 2.0 ** -19 + g.abs() * 2.0 ** -22) * h.abs() + TINY * (1 + u.abs())
    assert bool(((y - h).abs() <= tol).all())


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("n,k,cols", DENSE_LARGE)
def test_dense_large(M, n, k, cols, up):
    say("dense", n, k, cols, up)
    rng = np.random.default_rng(n * 7 + k + cols)
    q, s = integers(rng, (n, k)), scales(rng, n, 1 / np.sqrt(k) / 5000)
    w = integers(rng, (cols, k)), scales(rng, cols)
    w_up = (integers(rng, (cols, k)), scales(rng, cols)) if up else None
    check_large(M.int8_matmul((q, s), w, w_up=w_up), q, s, w, w_up)


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("N,E,K,k,cols", GROUPED_LARGE)
def test_grouped_large(M, N, E, K, k, cols, up):
    """Loads from none to half of the pairs, some pairs elsewhere; rows gathered where
    a token has more than one expert."""
    import torch
    gather = K > 1
    say("grouped", N, E, K, k, cols, gather, up)
    rng = np.random.default_rng(N + E + k)
    chance = np.array([0.0] + [2.0 ** -e for e in range(E - 1)] + [0.1])
    ids = rng.choice(E + 1, (N, K), p=chance / chance.sum())
    g = M.group_tokens(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    n = N if gather else N * K
    q, s = integers(rng, (n, k)), scales(rng, n, 1 / np.sqrt(k) / 5000)
    w = integers(rng, (E, cols, k)), scales(rng, (E, cols))
    w_up = (integers(rng, (E, cols, k)), scales(rng, (E, cols))) if up else None
    out = torch.full((N * K, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    M.int8_matmul((q, s), w, w_up=w_up, grouping=g, gather=gather, out=out)
    offsets, src = host(g.offsets), host(g.sorted_src)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        rows = torch.from_numpy(src[lo:hi] // K if gather else np.arange(lo, hi)).long().cuda()
        check_large(out[lo:hi], q[rows], s[rows], (w[0][e], w[1][e]),
                    None if w_up is None else (w_up[0][e], w_up[1][e]))
    assert bool((out[offsets[-1]:] == 7.0).all())


@pytest.mark.parametrize("rows,E,k,cols,up", [
    (16, 16, 4096, 4104, False), (16, 16, 4096, 2056, True), (4031, 64, 8192, 520, False),
    (9999, 200, 2560, 264, True), (30720, 384, 4096, 264, False), (6079, 64, 528, 4104, True),
    (42240, 384, 4096, 264, False), (24000, 200, 256, 4104, True)])
def test_many_experts_of_few_rows(M, rows, E, k, cols, up):
    """More weights than the memory-side cache holds, most experts in one tile."""
    import torch
    say("grouped", rows, E, k, cols, up)
    gen = torch.Generator(device="cuda").manual_seed(rows + k)

    def weight():
        return (torch.randint(-127, 128, (E, cols, k), generator=gen, device="cuda",
                              dtype=torch.int8),
                torch.rand(E, cols, generator=gen, device="cuda") + 0.5)
    w, w_up = weight(), weight() if up else None
    ids = torch.randint(0, E, (rows, 1), generator=gen, device="cuda", dtype=torch.int32)
    ids[rows // 2:rows // 2 + rows // 8] = E // 2    # one expert of several tiles
    g = M.group_tokens(ids, E)
    q = torch.randint(-127, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    s = (torch.rand(rows, generator=gen, device="cuda") + 0.5) / (5000 * k ** 0.5)
    y = M.int8_matmul((q, s), w, w_up=w_up, grouping=g)
    offsets = host(g.offsets)
    for e in {0, 1, E // 2, E // 3, E - 1}:
        lo, hi = offsets[e], offsets[e + 1]
        check_large(y[lo:hi], q[lo:hi], s[lo:hi], (w[0][e], w[1][e]),
                    None if w_up is None else (w_up[0][e], w_up[1][e]))

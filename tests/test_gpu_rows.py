"""GPU parity of the grouping and of the rows to the experts and back, with
their gradients, against the fp64 forms.

Tolerances.  U = 2^-24 is a rounding of fp32, HALF = 2^-8 half a step of bf16.
A sum over k adds at most K + 1 terms, each a product rounded once at most: (K +
2) U of the absolute terms.  A weight's gradient adds d products in a lane's d /
64 + 8 steps at most, six wave steps and four of a block: (d / 64 + 20) U of the
absolute products, one more for a kept row's value (code times scale).  A value
that leaves in bf16 adds HALF of it; a copied row has no error at all."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu

U, HALF, TINY = 2.0 ** -24, 2.0 ** -8, 1e-37


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


def tensor(a, dtype, offset=0):
    """offset > 0: that many elements into its storage (no 16-byte alignment)."""
    import torch
    a = torch.from_numpy(np.asarray(a, np.float32)).to(dtype)
    flat = torch.empty(a.numel() + offset, dtype=dtype, device="cuda")
    flat[offset:] = a.reshape(-1).cuda()
    return flat[offset:].view(a.shape)


def rand(rng, shape, std, dtype, offset=0):
    return tensor(std * rng.standard_normal(shape), dtype, offset)


def choice(rng, N, E, K, away):
    """K ids a token; away: none, some, all, one (every pair to one expert)."""
    import torch
    if away == "some":
        ids = rng.integers(-3, E + 4, (N, K))
    elif away == "all":
        ids = np.where(rng.random((N, K)) < 0.5, -1, E)
    elif away == "one":
        ids = np.full((N, K), E // 2)
    else:
        ids = np.argsort(rng.random((N, max(E, K))), axis=1)[:, :K] % E
    return torch.from_numpy(ids.astype(np.int32)).cuda()


GROUPS = [  # N, E, K, away
    (0, 3, 2, "none"), (1, 1, 1, "none"), (1, 384, 6, "none"), (1, 2, 8, "some"),
    (64, 384, 6, "none"), (37, 5, 3, "some"), (50, 7, 2, "all"), (300, 384, 8, "one"),
    (1365, 384, 6, "some"),      # 8190 pairs
    (1366, 384, 6, "none"),      # 8196 pairs
    (2731, 384, 6, "some"), (4097, 128, 8, "some"), (65537, 384, 8, "some"), (70001, 384, 1, "some"), (33000, 2, 4, "all"),
]


@pytest.mark.parametrize("N,E,K,away", GROUPS)
def test_group(M, N, E, K, away):
    import torch
    say("group", N, E, K, away)
    ids = choice(np.random.default_rng(N + E), N, E, K, away)
    g = M.group_tokens(ids, E)
    torch.cuda.synchronize()
    want = R.group(host(ids), E)
    for got, ref, name in zip((g.counts, g.offsets, g.sorted_src, g.src_pos), want,
                              ("counts", "offsets", "sorted_src", "src_pos")):
        assert np.array_equal(host(got), ref), name


def test_group_is_the_layers(M):
    """Without ids outside [0, E) the grouping is the one that forward uses."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    N, d, E, K, h = 700, 64, 24, 3, 32

    def w(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()
    W = M.ExpertWeights(w_router=w(E, d), w_gate=w(E, h, d), w_up=w(E, h, d), w_down=w(E, d, h))
    _, aux = M.forward(w(N, d), W, K, aux=("topk_ids", "counts", "offsets", "sorted_src", "src_pos"))
    grouping = M.group_tokens(aux["topk_ids"], E)
    for n in ("counts", "offsets", "sorted_src", "src_pos"):
        assert torch.equal(getattr(grouping, n), aux[n]), n


ROWS = [  # N, d, E, K, type, away, offset
    (1, 2560, 384, 6, "bf16", "none", 0),
    (1, 1, 2, 1, "bf16", "none", 0),
    (3, 1, 4, 8, "f32", "some", 0),
    (64, 2560, 384, 6, "bf16", "some", 0),
    (33, 777, 10, 5, "bf16", "some", 0),
    (33, 777, 10, 5, "f32", "some", 0),
    (129, 264, 7, 7, "bf16", "none", 0),
    (129, 264, 7, 7, "bf16", "some", 1),     # not aligned: element by element
    (40, 8192, 3, 2, "f32", "none", 0),
    (40, 8192, 3, 2, "bf16", "one", 0),
    (17, 128, 9, 4, "f32", "all", 0),
    (260, 516, 11, 8, "f32", "some", 1),
    (4100, 72, 20, 3, "bf16", "some", 0),
    # about one piece of eight (four) elements, and a piece more than a block's
    (19, 7, 4, 2, "bf16", "some", 0), (19, 8, 4, 2, "bf16", "some", 1),
    (19, 9, 4, 2, "bf16", "none", 0), (19, 15, 4, 3, "bf16", "some", 0),
    (19, 3, 4, 2, "f32", "some", 0), (19, 4, 4, 2, "f32", "none", 1),
    (19, 5, 4, 6, "f32", "some", 0), (19, 7, 4, 8, "f32", "some", 0),
    (11, 1025, 4, 2, "bf16", "some", 0), (11, 1023, 4, 2, "f32", "some", 1),
    (11, 2049, 4, 2, "bf16", "some", 0), (11, 8191, 4, 3, "f32", "some", 0),
]


def setup(seed, N, d, E, K, kind, away, offset):
    import torch
    rng = np.random.default_rng(seed)
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    ids = choice(rng, N, E, K, away)
    return rng, dtype, R.group(host(ids), E), ids


@pytest.mark.parametrize("case", ROWS)
def test_permute_and_gradient(M, case):
    import torch
    N, d, E, K, kind, away, offset = case
    say("permute", case)
    rng, dtype, (_, offsets, src, pos), ids = setup(7, *case)
    g = M.group_tokens(ids, E)
    x = rand(rng, (N, d), 1.0, dtype, offset)
    out = rand(rng, (N * K, d), 5.0, dtype, offset)
    held = f64(out)
    rows = M.permute(x, g, out=out)
    assert rows.data_ptr() == out.data_ptr()
    assert np.array_equal(f64(rows), R.permute(f64(x), src, K, held))
    if away != "all":
        fresh = M.permute(x, g)
        n = int(offsets[-1])
        assert torch.equal(fresh[:n], rows[:n])
    grad = rand(rng, (N * K, d), 1e-2, dtype, offset)
    if offsets[-1] < N * K:
        grad[int(offsets[-1]):] = float("nan")   # rows without a pair are not read
    dx = M.permute_backward(grad, g)
    want, mag = R.unpermute(np.nan_to_num(f64(grad)), pos)
    half = U if kind == "f32" else HALF
    assert dx.dtype == dtype
    assert np.all(np.abs(f64(dx) - want) <= (K + 2) * U * mag + half * np.abs(want) + TINY)


@pytest.mark.parametrize("weighted,based", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("case", ROWS)
def test_unpermute(M, case, weighted, based):
    N, d, E, K, kind, away, offset = case
    import torch
    say("unpermute", case, weighted, based)
    rng, dtype, (_, offsets, src, pos), ids = setup(8, *case)
    g = M.group_tokens(ids, E)
    rows = rand(rng, (N * K, d), 1.0, dtype, offset)
    rows[int(offsets[-1]):] = float("nan")
    w = rand(rng, (N, K), 1.0, torch.float32) if weighted else None
    base = rand(rng, (N, d), 2.0, dtype, offset) if based else None
    y, kept = M.unpermute(rows, g, weights=w, base=base)
    assert kept is None and y.dtype == dtype
    want, mag = R.unpermute(np.nan_to_num(f64(rows)), pos, None if w is None else f64(w),
                            None if base is None else f64(base))
    half = U if kind == "f32" else HALF
    assert np.all(np.abs(f64(y) - want) <= (K + 2) * U * mag + half * np.abs(want) + TINY)


@pytest.mark.parametrize("case", ROWS)
def test_unpermute_backward(M, case):
    N, d, E, K, kind, away, offset = case
    import torch
    say("unpermute backward", case)
    rng, dtype, (_, offsets, src, pos), ids = setup(9, *case)
    g = M.group_tokens(ids, E)
    dy = rand(rng, (N, d), 1.0, dtype, offset)
    rows = rand(rng, (N * K, d), 1.0, dtype, offset)
    rows[int(offsets[-1]):] = float("nan")
    w = rand(rng, (N, K), 1.0, torch.float32)
    out = rand(rng, (N * K, d), 5.0, dtype, offset)
    held = f64(out)
    half = U if kind == "f32" else HALF
    for weights, r in ((w, rows), (None, rows), (w, None)):
        out.copy_(tensor(held, dtype))
        got, dw = M.unpermute_backward(dy, g, weights=weights, rows=r, out=out)
        drows, want, mag = R.unpermute_backward(f64(dy), pos,
                                                None if weights is None else f64(weights),
                                                None if r is None else np.nan_to_num(f64(r)), held)
        n = int(offsets[-1])
        assert np.all(np.abs(f64(got)[:n] - drows[:n]) <= (U + half) * np.abs(drows[:n]) + TINY)
        assert np.array_equal(f64(got)[n:], held[n:])
        if r is None:
            assert dw is None
        else:
            assert np.all(np.abs(f64(dw) - want) <= (d / 64 + 20) * U * mag + TINY)
            assert np.all(f64(dw)[pos < 0] == 0)


KEPT = [  # N, d, E, K, away
    (1, 128, 2, 1, "none"), (1, 2560, 384, 6, "none"), (64, 2560, 48, 6, "some"),
    (70, 384, 5, 8, "one"), (33, 8192, 4, 3, "some"), (700, 256, 20, 4, "none"),
    (19, 640, 3, 5, "all"),
]


def values(codes, scales):
    import torch
    v = host(codes.view(torch.float8_e4m3fn).float()).astype(np.float64)
    return v * np.repeat(f64(scales), 128, axis=1)


@pytest.mark.parametrize("N,d,E,K,away", KEPT)
def test_rows_kept_in_8_bits(M, N, d, E, K, away):
    import torch
    say("kept", N, d, E, K, away)
    rng, _, (_, offsets, src, pos), ids = setup(11, N, d, E, K, "bf16", away, 0)
    n = int(offsets[-1])
    g = M.group_tokens(ids, E)
    bf = torch.bfloat16
    # the tokens' codes and the experts' inputs from them
    x = rand(rng, (N, d), 1.0, bf)
    x[:, 5] *= 40
    x[0, :128] = 0
    q = M.fp8_quantize_rows(x)
    out = torch.full((N * K, d), 3.0, dtype=bf, device="cuda")
    rows = M.permute(q, g, out=out)
    want = R.permute(values(*q), src, K, np.full((N * K, d), 3.0))
    assert rows.dtype == bf
    assert np.all(np.abs(f64(rows) - want) <= (U + HALF) * np.abs(want) + TINY)
    # the codes that unpermute leaves are the row quantiser's
    r = rand(rng, (N * K, d), 1.0, bf)
    r[0] = 0
    w, base = rand(rng, (N, K), 1.0, torch.float32), rand(rng, (N, d), 1.0, bf)
    y, kept = M.unpermute(r, g, weights=w, base=base, checkpoint=True)
    y0, _ = M.unpermute(r, g, weights=w, base=base)
    assert torch.equal(y, y0)
    codes, scales = M.fp8_quantize_rows(r)
    assert torch.equal(kept[0][:n], codes[:n]) and torch.equal(kept[1][:n], scales[:n])
    # gradients from them
    dy = rand(rng, (N, d), 1.0, bf)
    kept[1][n:] = float("nan")
    drows, dw = M.unpermute_backward(dy, g, weights=w, rows=kept)
    v = values(codes, scales)
    _, want, mag = R.unpermute_backward(f64(dy), pos, f64(w), v, np.zeros((N * K, d)))
    assert np.all(np.abs(f64(dw) - want) <= (d / 64 + 21) * U * mag + TINY)
    plain, _ = M.unpermute_backward(dy, g, weights=w, rows=r)
    assert torch.equal(drows[:n], plain[:n])


def test_kept_codes_of_every_significand(M):
    """The codes that unpermute leaves are the row quantiser's, bit for bit: every
    significand of a group's largest value against every significand of its others,
    over the E4M3 range and below, at exponents down to where the scale is
    subnormal."""
    import torch
    sig = torch.arange(128, 256, device="cuda").double() / 128
    for e in (-126, -100, -61, -59, 0, 40, 119):
        groups = []
        for shift in range(0, 20):
            other = torch.ldexp(sig, torch.tensor(-shift, device="cuda"))
            m = torch.where(torch.arange(128, device="cuda") % 2 == 1, -other, other).repeat(128, 1)
            m[:, 0] = sig * 2      # the group's largest value
            groups.append(m)
        rows = torch.ldexp(torch.cat(groups, 1), torch.tensor(e, device="cuda")).bfloat16()
        N = rows.shape[0]
        g = M.group_tokens(torch.zeros(N, 1, dtype=torch.int32, device="cuda"), 2)
        _, kept = M.unpermute(rows, g, checkpoint=True)
        codes, scales = M.fp8_quantize_rows(rows)
        assert torch.equal(kept[1], scales) and torch.equal(kept[0], codes), e


def test_kept_codes_of_infinities(M):
    """Groups with an infinity or a NaN: the row quantiser's codes and scales there too."""
    import torch
    rng = np.random.default_rng(5)
    rows = torch.from_numpy(rng.standard_normal((6, 384)).astype(np.float32)).cuda().bfloat16()
    rows[0, 3], rows[1, 200], rows[2, 383] = float("inf"), float("-inf"), float("nan")
    rows[3, 0], rows[3, 1] = float("inf"), float("nan")
    g = M.group_tokens(torch.zeros(6, 1, dtype=torch.int32, device="cuda"), 2)
    _, kept = M.unpermute(rows, g, checkpoint=True)
    codes, scales = M.fp8_quantize_rows(rows)
    assert torch.equal(kept[0], codes)
    assert torch.equal(kept[1].view(torch.int32) & 0x7FC00000, scales.view(torch.int32) & 0x7FC00000)
    finite = torch.isfinite(scales)
    assert int(finite.sum()) == 14 and torch.equal(kept[1][finite], scales[finite])


def test_gradients_against_differences(M):
    """fp32 rows: (L(w + h) - L(w - h)) / 2h of L = <dy, y>, which is linear in
    every argument, so only roundings separate the two: 2 (K + 2) U of the terms
    of y times dy, over 2h."""
    import torch
    rng, dtype, (_, offsets, src, pos), ids = setup(13, 23, 200, 6, 4, "f32", "some", 0)
    N, d, K = 23, 200, 4
    g = M.group_tokens(ids, 6)
    rows, dy = rand(rng, (N * K, d), 1.0, dtype), rand(rng, (N, d), 1.0, dtype)
    w = rand(rng, (N, K), 1.0, dtype)
    drows, dw = M.unpermute_backward(dy, g, weights=w, rows=rows)
    h = 0.5
    term = np.zeros((N, K))
    for t in range(N):
        for k in range(K):
            up, dn = w.clone(), w.clone()
            up[t, k] += h
            dn[t, k] -= h
            yu, yd = f64(M.unpermute(rows, g, weights=up)[0]), f64(M.unpermute(rows, g, weights=dn)[0])
            num = np.sum(f64(dy) * (yu - yd)) / (2 * h)
            _, mag = R.unpermute(f64(rows), pos, np.abs(f64(w)) + h)
            tol = 2 * (K + 3) * U * np.sum(np.abs(f64(dy)[t]) * mag[t]) / (2 * h) + \
                (d / 64 + 20) * U * np.sum(np.abs(f64(dy)[t])) * np.abs(f64(rows)).max()
            assert abs(num - f64(dw)[t, k]) <= tol, (t, k)


@pytest.mark.parametrize("width", [256, 11, 261, 5])
def test_infinities_and_nan_stay_where_they_are(M, width):
    """A NaN or infinity in a row reaches its own token only, also with a weight
    of zero next to it; rows without a pair reach none."""
    import torch
    N, d, E, K = 6, width, 3, 2
    ids = torch.tensor([[0, 1], [1, 2], [-1, 0], [2, 2], [-1, -1], [1, 0]], dtype=torch.int32).cuda()
    g = M.group_tokens(ids, E)
    pos = host(g.src_pos)
    for dtype in (torch.bfloat16, torch.float32):
        rows = torch.ones(N * K, d, dtype=dtype, device="cuda")
        rows[int(pos[1, 0]), 3] = float("nan")
        rows[int(pos[3, 1]), 4] = float("inf")
        rows[int(host(g.offsets)[-1]):] = float("nan")
        y, _ = M.unpermute(rows, g)
        y = f64(y)
        assert np.isnan(y[1, 3]) and np.isinf(y[3, 4])
        y[1, 3] = y[3, 4] = 0
        assert np.all(np.isfinite(y)) and np.all(y[4] == 0)
        dy = torch.ones(N, d, dtype=dtype, device="cuda")
        _, dw = M.unpermute_backward(dy, g, rows=rows)
        dw = f64(dw)
        assert np.isnan(dw[1, 0]) and np.isinf(dw[3, 1])
        dw[1, 0] = dw[3, 1] = 0
        assert np.all(np.isfinite(dw)) and np.all(dw[4] == 0)
    if d != 256:
        return
    rows = torch.ones(N * K, d, dtype=torch.bfloat16, device="cuda")
    rows[int(pos[1, 0]), 3] = float("nan")
    rows[int(pos[3, 1]), 200] = float("-inf")
    _, (codes, scales) = M.unpermute(rows, g, checkpoint=True)
    s = f64(scales)
    assert np.isnan(s[pos[1, 0], 0]) and np.isinf(s[pos[3, 1], 1])
    n = int(host(g.offsets)[-1])
    assert np.sum(~np.isfinite(s[:n])) == 2


def test_places_out_of_range_touch_nothing(M):
    """A place outside [0, N*K) is no place, whatever it is."""
    import torch
    N, d, K = 4, 64, 2
    pos = torch.tensor([[0, 8], [1 << 30, 3], [-5, 4], [-(1 << 31), 7]], dtype=torch.int32).cuda()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = M.Grouping(none, none, none, pos)
    x = torch.arange(N, device="cuda").float().unsqueeze(1).expand(N, d).contiguous() + 1
    out = torch.zeros(N * K, d, device="cuda")
    rows = M.permute(x, g, out=out)
    assert host(rows[:, 0]).tolist() == [1, 0, 0, 2, 3, 0, 0, 4]
    y, _ = M.unpermute(rows, g)
    assert host(y[:, 5]).tolist() == [1, 2, 3, 4]


def test_rows_past_four_gigabytes(M):
    """Places whose rows lie past 2^32 bytes."""
    import torch
    N, d, K, E = 40000, 8192, 4, 5          # 5.2 GB of fp32 rows
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, E, (N, K), generator=gen, device="cuda", dtype=torch.int32)
    g = M.group_tokens(ids, E)
    x = torch.randn(N, d, generator=gen, device="cuda")
    rows = M.permute(x, g)
    pick = torch.arange(0, N * K, 997, device="cuda")
    tok = g.sorted_src[pick].long() // K
    assert torch.equal(rows[pick], x[tok])
    assert torch.equal(rows[-1], x[g.sorted_src[-1].long() // K])
    w = torch.rand(N, K, generator=gen, device="cuda")
    y, _ = M.unpermute(rows, g, weights=w)
    t = torch.arange(0, N, 991, device="cuda")
    ref = x[t].double() * w[t].double().sum(1, keepdim=True)
    assert bool(((y[t].double() - ref).abs() <= (K + 2) * U * ref.abs() + TINY).all())
    del y
    drows, dw = M.unpermute_backward(x, g, weights=w, rows=rows)
    ref = (x[t].double() ** 2).sum(1, keepdim=True).expand(-1, K)
    assert bool(((dw[t].double() - ref).abs() <= (d / 64 + 20) * U * ref).all())
    p = g.src_pos[t].long().reshape(-1)
    ref = (x[t].unsqueeze(1) * w[t].unsqueeze(2)).reshape(-1, d)
    assert torch.equal(drows[p], ref)


def test_calls_are_repeatable_and_take_streams(M):
    import torch
    N, d, E, K = 1000, 640, 12, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(-1, E, (N, K), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.randn(N, d, generator=gen, device="cuda").bfloat16()
    w = torch.rand(N, K, generator=gen, device="cuda")

    def chain(stream=None):
        g = M.group_tokens(ids, E, stream=stream)
        out = torch.zeros(N * K, d, dtype=x.dtype, device="cuda") if stream is None else zeros
        rows = M.permute(x, g, out=out, stream=stream)
        y, kept = M.unpermute(rows, g, weights=w, base=x, checkpoint=True, stream=stream)
        drows, dw = M.unpermute_backward(y, g, weights=w, rows=kept, out=rows.clone() if stream is None else zeros2,
                                         stream=stream)
        return y, dw, M.permute_backward(drows, g, stream=stream)
    zeros = torch.zeros(N * K, d, dtype=x.dtype, device="cuda")
    zeros2 = torch.zeros(N * K, d, dtype=x.dtype, device="cuda")
    first = chain()
    for a, b in zip(first, chain()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, got):
        assert torch.equal(a, b)


def test_refusals(M):
    import torch
    N, d, E, K = 4, 128, 3, 2
    ids = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    g = M.group_tokens(ids, E)
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(N * K, d, dtype=torch.bfloat16, device="cuda")
    q = M.fp8_quantize_rows(x)
    f32 = torch.zeros(N, K, device="cuda")
    bad = [
        (ValueError, lambda: M.group_tokens(ids[0], E)),
        (TypeError, lambda: M.group_tokens(ids.long(), E)),
        (TypeError, lambda: M.group_tokens(ids.cpu(), E)),
        (M.MoeError, lambda: M.group_tokens(ids, 385)),
        (ValueError, lambda: M.permute(x[:3], g)),
        (TypeError, lambda: M.permute(x.half(), g)),
        (TypeError, lambda: M.permute(x, g, out=rows.float())),
        (ValueError, lambda: M.permute(x, g, out=rows[:-1])),
        (ValueError, lambda: M.permute((q[0][:3], q[1][:3]), g)),
        (ValueError, lambda: M.permute((q[0], None), g)),
        (ValueError, lambda: M.permute((q[0], q[1].t()), g)),
        (ValueError, lambda: M.permute(x.t(), M.Grouping(None, None, None, torch.zeros(d, 1, dtype=torch.int32, device="cuda")))),
        (ValueError, lambda: M.permute_backward(x, g)),
        (ValueError, lambda: M.unpermute(x, g)),
        (ValueError, lambda: M.unpermute(rows, g, weights=f32[:2])),
        (TypeError, lambda: M.unpermute(rows, g, base=x.float())),
        (M.MoeError, lambda: M.unpermute(rows.float(), g, checkpoint=True)),
        (M.MoeError, lambda: M.unpermute(rows[:, :64].contiguous(), g, checkpoint=True)),
        (ValueError, lambda: M.unpermute_backward(rows, g)),
        (TypeError, lambda: M.unpermute_backward(x, g, rows=rows.float())),
        (ValueError, lambda: M.unpermute_backward(x, g, rows=q)),
        (M.MoeError, lambda: M.unpermute_backward(x.float(), g, rows=M.fp8_quantize_rows(rows))),
        (M.MoeError, lambda: M.unpermute_backward(x, g, rows=rows, out=rows)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("E", [1, 7, 384])
@pytest.mark.parametrize("pairs", [1023, 1024, 1025, 2048, 8191, 8192, 8193, 16385, 24575, 24576,
                                   24577, 30000])
def test_group_around_the_blocks(M, pairs, E):
    """Numbers of pairs around those of a block, of a thread's loads at once and of the
    one launch; loads even, one expert's alone, and ids far out of range."""
    import torch
    rng = np.random.default_rng(pairs + E)
    for kind in range(3):
        ids = rng.integers(-1, E + 1, (pairs, 1))
        if kind == 1:
            ids[:] = E - 1
        if kind == 2:
            ids[rng.random((pairs, 1)) < 0.3] = rng.choice([2 ** 31 - 1, -2 ** 31, E])
        t = torch.from_numpy(ids.astype(np.int32)).cuda()
        g = M.group_tokens(t, E)
        want = R.group(ids, E)
        got = (g.counts, g.offsets, g.sorted_src, g.src_pos)
        for a, b in zip(got, want):
            assert np.array_equal(host(a).ravel(), np.asarray(b).ravel()), (pairs, E, kind)

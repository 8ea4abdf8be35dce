"""8-bit integer products whose rows are picked from the largest a that is taken, 4 GiB -
512 KiB: offsets past 2^31 and the last row, in a few-row form and in a form of tiles.

Tolerance: the sums are exact; their conversion, the product of the scales and its
product with the sum round once each, 3 x 2^-24, and bf16 half a step, 2^-8."""
import ctypes as C

import pytest

pytestmark = pytest.mark.gpu

N, DEPTH, K = 65528, 65536, 2


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


@pytest.fixture(scope="module")
def tokens(M):
    """Zeros but for a few rows on both sides of 2 GiB and at the end."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    a = torch.zeros(N, DEPTH, dtype=torch.int8, device="cuda")
    live = torch.tensor([0, 1, 32767, 32768, 32769, 50000, N - 2, N - 1], device="cuda")
    a[live] = torch.randint(-128, 128, (len(live), DEPTH), generator=gen, device="cuda").to(torch.int8)
    yield a, torch.rand(N, generator=gen, device="cuda") / 1e4 + 1e-5, live
    del a
    torch.cuda.empty_cache()


# one column group of 16 rows or fewer: the few-row form; thousands of rows: tiles
@pytest.mark.parametrize("rows,cols,up", [(1, 8, False), (13, 8, True), (3000, 520, False),
                                          (3000, 520, True)])
def test_rows_picked_from_four_gigabytes(M, tokens, rows, cols, up):
    import torch
    from sigmoid_top_routing_router_amd import _lib
    lib = _lib.load()
    print(f"[gathered] rows={rows} cols={cols} up={up}", flush=True)
    a, sa, live = tokens
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    E, split = 2, rows // 3
    offsets = torch.tensor([0, split, rows], dtype=torch.int32, device="cuda")
    pick = torch.randint(0, len(live), (rows,), generator=gen, device="cuda")
    pick[0] = pick[-1] = len(live) - 1
    src = (live[pick] * K + torch.randint(0, K, (rows,), generator=gen, device="cuda")).int()

    def weight():
        return (torch.randint(-128, 128, (E, cols, DEPTH), generator=gen, device="cuda").to(torch.int8),
                torch.rand(E, cols, generator=gen, device="cuda") / 1e2 + 1e-3)
    w, u = weight(), weight() if up else (None, None)
    out = torch.full((rows + 1, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    p = _lib.MoeInt8Matmul(N, rows, DEPTH, cols, E, K,
                           *[None if t is None else t.data_ptr()
                             for t in (a, sa, *w, *u, offsets, src)])
    _lib.check(lib.moe_int8_matmul(C.byref(p), out.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert bool((out[rows] == 7).all())

    def products(w):
        """Every live row with both weights, in 64 bits."""
        x = a[live].double()
        return torch.stack([x @ w[0][e].double().t().contiguous() * sa[live].double()[:, None]
                            * w[1][e].double() for e in range(E)])
    expert = (torch.arange(rows, device="cuda") >= split).long()
    g = products(w)[expert, pick]
    got = out[:rows].double()
    half, one = 2.0 ** -8, 2.0 ** -24
    if not up:
        assert bool(((got - g).abs() <= (3.1 * one + half) * g.abs()).all())
        return
    # as in the other tests of silu(g) u: |g| 2^-22 + 2^-19 of it
    h = g * torch.sigmoid(g) * products(u)[expert, pick]
    assert bool(((got - h).abs() <= (half + 2.0 ** -19 + g.abs() * 2.0 ** -22) * h.abs()
                 + 1e-35 * (1 + h.abs())).all())

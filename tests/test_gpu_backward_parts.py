"""grad_x of moe_backward is rounded where the header says and nowhere else: its
parts (a pair's, the shared expert's and the router's) are summed in fp32.

Per value: dG, dU and, with a router, grad_logits_out are rounded to bf16 once
(HALF = 2^-8 of a term) and the result once; fp32 sums as in
test_gpu_backward: (HALF 1.01 + 2 C + 2^-17) mag + HALF |out|.

Pooled: the fp64 form with just these roundings is off by `stated`, with a
rounding of every pair's part to bf16 more by `more`, some 1.2 times as much.
Both are sums over 10^5 and more independent roundings, so each is known to one
part in 300, and fp32 sums move a rounding in some 2^-24 / 2^-9 C of all values:
the kernel's error is `stated` within one per cent and has to lie below the
geometric mean of the two."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O
from tests.gpu_util import rel_l2, say
from tests.test_gpu_backward import HALF, f64, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def bf16(v):
    return O.bf16_to_f32(O.f32_to_bf16_rne(v.astype(np.float32))).astype(np.float64)


def rows_part(f, t, s, names, e):
    """dG W_g + dU W_u of one expert's rows, dG and dU in bf16."""
    wg, wu, wd = (f[n][e].astype(np.float64) for n in names)
    x, dy = f["x"][t].astype(np.float64), f["dy"][t].astype(np.float64)
    G, U, Q = x @ wg.T, x @ wu.T, dy @ wd
    sg = 1.0 / (1.0 + np.exp(-G))
    dU, dG = s[:, None] * Q * G * sg, s[:, None] * Q * U * sg * (1 + G * (1 - sg))
    return bf16(dG) @ wg + bf16(dU) @ wu


@pytest.mark.parametrize("N,d,E,K,h,hs,router", [(600, 512, 12, 8, 96, 0, False),
                                                 (300, 1024, 9, 4, 64, 0, True),
                                                 (500, 320, 16, 6, 64, 32, True)])
def test_parts_of_grad_x_are_not_rounded(M, N, d, E, K, h, hs, router):
    say("backward, parts of grad_x", N, d, E, K, h, hs, router)
    L, Z, ids = make(31 + N, N, d, E, K, h, hs, router=router)
    f = {k: O.bf16_to_f32(v) for k, v in L.items()}
    shared = tuple(f[k][0] for k in ("ws_gate", "ws_up", "ws_down")) if hs else None
    want, mag = B.layer_backward(f["x"], f["dy"], Z, ids, f.get("w_router"), f["w_gate"], f["w_up"],
                                 f["w_down"], shared)
    got = f64(run(M, L, Z, ids)[0])
    c = (max(N, d, h, E, hs) / 16 + 20) * 2.0 ** -24
    tol = (HALF * 1.01 + 2 * c + 2.0 ** -17) * mag["x"] + HALF * np.abs(want["x"]) + 1e-37
    assert np.all(np.abs(got - want["x"]) <= tol)

    stated, more = np.zeros((N, d)), np.zeros((N, d))
    for e in range(E):
        t, k = np.nonzero(ids == e)
        s = 1.0 / (1.0 + np.exp(-Z[t, e].astype(np.float64)))
        part = rows_part(f, t, s, ("w_gate", "w_up", "w_down"), e)
        np.add.at(stated, t, part)
        np.add.at(more, t, bf16(part))
    rest = np.zeros((N, d))
    if hs:
        rest += rows_part(f, np.arange(N), np.ones(N), ("ws_gate", "ws_up", "ws_down"), 0)
    if router:
        rest += bf16(want["logits"]) @ f["w_router"].astype(np.float64)
    stated, more = (rel_l2(bf16(v + rest), want["x"]) for v in (stated, more))
    own = rel_l2(got, want["x"])
    say("off by", f"{own:.3e}", "stated", f"{stated:.3e}", "parts rounded", f"{more:.3e}")
    assert more > 1.1 * stated
    assert own < (stated * more) ** 0.5

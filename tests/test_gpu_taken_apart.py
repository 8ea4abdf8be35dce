"""The operators that take the layer apart, used together: the layer rebuilt from
them, its gradients, experts in 8-bit integers, and both captured into graphs.

The rebuilt layer rounds where the layer does (the hidden rows and the experts'
rows to bf16, 2^-8 of the value each), so that the two differ by the order of fp32
sums and by roundings that fall the other way: each of the two roundings by at most
a whole step, 2^-7 of a row's values, and the layer's own half-steps; relative to
the output's norm 3 2^-8 bounds both (errors of different elements are
independent, the bound takes them as if they all had one sign).  Gradients chain
three more roundings of 2^-8: 6 2^-8.  Weights and tokens in 8 bits (E4M3, half a
step 2^-4 at most a value, a third of it on average over a binade's values) add
2^-4 for each operand; integers half a step of amax / 127 each."""
import pytest

pytestmark = pytest.mark.gpu

B = 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def layer(M, seed, N=600, d=256, E=12, K=3, h=96):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def w(std, *s):
        return (std * torch.randn(*s, generator=g, device="cuda")).bfloat16()
    W = M.ExpertWeights(w_router=w(d ** -0.5, E, d), w_gate=w(d ** -0.5, E, h, d),
                        w_up=w(d ** -0.5, E, h, d), w_down=w(h ** -0.5, E, d, h),
                        ws_gate=w(d ** -0.5, 1, h, d), ws_up=w(d ** -0.5, 1, h, d),
                        ws_down=w(h ** -0.5, 1, d, h))
    return W, w(1.0, N, d), w(1.0, N, d)


def experts(rows, offsets, W):
    """Every expert's rows through its SwiGLU (fp32 products, rounded as the layer
    does): rows [P, d], offsets on the host.  Returns what backward needs too."""
    import torch
    hid = torch.empty(rows.shape[0], W.w_gate.shape[1], dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(rows)
    for e in range(W.w_gate.shape[0]):
        s = slice(offsets[e], offsets[e + 1])
        x = rows[s].float()
        gate, up = x @ W.w_gate[e].float().t(), x @ W.w_up[e].float().t()
        hid[s] = (torch.nn.functional.silu(gate) * up).bfloat16()
        out[s] = (hid[s].float() @ W.w_down[e].float().t()).bfloat16()
    return out


def shared(x, W):
    import torch
    gate, up = x.float() @ W.ws_gate[0].float().t(), x.float() @ W.ws_up[0].float().t()
    hid = (torch.nn.functional.silu(gate) * up).bfloat16()
    return (hid.float() @ W.ws_down[0].float().t()).bfloat16()


def test_layer_rebuilt(M):
    W, x, _ = layer(M, 1)
    E, K = 12, 3
    y, aux = M.forward(x, W, K, aux=("topk_ids", "topk_weights", "offsets"))
    g = M.group_tokens(aux["topk_ids"], E)
    rows = M.permute(x, g)
    out = experts(rows, g.offsets.tolist(), W)
    y2, kept = M.unpermute(out, g, weights=aux["topk_weights"], base=shared(x, W), checkpoint=True)
    assert rel(y2, y) <= 3 * B
    codes, scales = M.fp8_quantize_rows(out)
    assert bool((kept[0] == codes).all()) and bool((kept[1] == scales).all())


@pytest.mark.parametrize("keep", [False, True])
def test_training_step_against_the_layers(M, keep):
    """Gradients of x, of the logits and of the experts' weights through the pieces,
    against moe_backward's of the same layer without router and shared expert.  With
    keep, the tokens and the experts' rows come back from 8 bits."""
    import torch
    W, x, dy = layer(M, 2)
    E, K = 12, 3
    R = M.ExpertWeights(w_router=None, w_gate=W.w_gate, w_up=W.w_up, w_down=W.w_down)
    z = x.float() @ W.w_router.float().t()
    _, aux = M.forward(x, R, K, logits_in=z, aux=("topk_ids", "topk_weights"))
    ids, s = aux["topk_ids"], aux["topk_weights"]
    dx, dz, grads = M.backward(dy, x, R, z, ids)

    g = M.group_tokens(ids, E)
    off = g.offsets.tolist()
    # forward: what is kept for the way back
    out = experts(M.permute(x, g), off, R)
    _, kept = M.unpermute(out, g, weights=s, checkpoint=keep)
    x_kept = M.fp8_quantize_rows(x) if keep else x
    rows_kept = kept if keep else out
    # backward
    drows, ds = M.unpermute_backward(dy, g, weights=s, rows=rows_kept)
    rows = M.permute(x_kept, g)
    drow_x = torch.empty_like(rows)
    gw = [torch.empty_like(w) for w in (R.w_gate, R.w_up, R.w_down)]
    for e in range(E):
        c = slice(off[e], off[e + 1])
        leaf = [t.float().requires_grad_() for t in (rows[c], R.w_gate[e], R.w_up[e], R.w_down[e])]
        hid = torch.nn.functional.silu(leaf[0] @ leaf[1].t()) * (leaf[0] @ leaf[2].t())
        got = torch.autograd.grad(hid @ leaf[3].t(), leaf, drows[c].float())
        drow_x[c] = got[0].bfloat16()
        for w, t in zip(gw, got[1:]):
            w[e] = t.bfloat16()
    dx2 = M.permute_backward(drow_x, g)
    dz2 = torch.zeros_like(z)
    dz2.scatter_(1, ids.long(), ds * s * (1 - s))
    far = 6 * B + (2.0 ** -3 if keep else 0.0)
    assert rel(dx2, dx) <= far and rel(dz2, dz) <= far
    for a, b in zip(gw, (grads.w_gate, grads.w_up, grads.w_down)):
        assert rel(a, b) <= far


def test_experts_in_integers(M):
    """Sorted tokens, both products in 8 bits, back: against the same layer with
    bf16 experts.  An operand's half step is amax / 254 (a normal row's amax is 3 to 4
    of its spread: 2^-6 of the spread, 2^-6.8 of it on average); two products with two
    operands each: 4 2^-6."""
    import torch
    W, x, _ = layer(M, 3)
    E, K = 12, 3
    R = M.ExpertWeights(w_router=W.w_router, w_gate=W.w_gate, w_up=W.w_up, w_down=W.w_down)
    y, aux = M.forward(x, R, K, aux=("topk_ids", "topk_weights"))
    wg, wu, wd = (M.int8_quantize_rows(t) for t in (W.w_gate, W.w_up, W.w_down))
    g = M.group_tokens(aux["topk_ids"], E)

    def run():
        hid = M.int8_matmul(M.int8_quantize_rows(x), wg, w_up=wu, grouping=g, gather=True)
        out = M.int8_matmul(M.int8_quantize_rows(hid), wd, grouping=g)
        return M.unpermute(out, g, weights=aux["topk_weights"])[0]
    y2 = run()
    assert rel(y2, y) <= 2.0 ** -4
    # the tokens sorted first give the same bits
    xs = M.permute(x, g)
    hid = M.int8_matmul(M.int8_quantize_rows(xs), wg, w_up=wu, grouping=g)
    assert torch.equal(hid, M.int8_matmul(M.int8_quantize_rows(x), wg, w_up=wu, grouping=g, gather=True))


def test_step_in_a_graph(M):
    """Forward and backward of the pieces captured, replayed with other inputs and
    other groupings, the program's own eager calls between the replays."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    N, d, E, K = 900, 384, 16, 4
    x = torch.empty(N, d, dtype=torch.bfloat16, device="cuda")
    dy, s = torch.empty_like(x), torch.empty(N, K, device="cuda")
    ids = torch.empty(N, K, dtype=torch.int32, device="cuda")
    rows, back = (torch.zeros(N * K, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def fill():
        for t in (x, dy):
            t.normal_(generator=gen)
        s.uniform_(generator=gen)
        ids.random_(-2, E + 2, generator=gen)

    def step():
        rows.zero_()
        back.zero_()
        g = M.group_tokens(ids, E)
        M.permute(x, g, out=rows)
        y, kept = M.unpermute(rows, g, weights=s, base=x, checkpoint=True)
        _, ds = M.unpermute_backward(dy, g, weights=s, rows=kept, out=back)
        return y, ds, M.permute_backward(back, g), g.offsets, back
    fill()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        fill()
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), i

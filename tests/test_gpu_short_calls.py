"""The short way to the small calls (the binding's extension module) against the way
through Python, which a given stream takes: the same results, outputs and refusals."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def state(M, N=37, E=6, K=3, d=256, dtype=None, seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = dtype or torch.bfloat16

    def rand(*shape, t=dtype):
        return torch.randn(*shape, generator=gen, device="cuda").to(t)
    ids = torch.randint(-1, E, (N, K), generator=gen, device="cuda", dtype=torch.int32)
    return {"ids": ids, "E": E, "x": rand(N, d), "rows": rand(N * K, d), "base": rand(N, d),
            "w": rand(N, K, t=torch.float32), "we": rand(E, 40, d, t=torch.bfloat16),
            "wu": rand(E, 40, d, t=torch.bfloat16)}


def all_calls(M, s, stream=None):
    """Every call, outputs given so that rows without a pair hold the same."""
    import torch
    N, d = s["x"].shape
    P = s["rows"].shape[0]
    g = M.group_tokens(s["ids"], s["E"], stream=stream)
    held = lambda t=None, c=d: torch.full((P, c), 7, dtype=t or s["x"].dtype, device="cuda")
    out = [g.counts, g.offsets, g.sorted_src, g.src_pos]
    out += [M.permute(s["x"], g, out=held(), stream=stream),
            M.permute_backward(s["rows"], g, stream=stream),
            M.unpermute(s["rows"], g, stream=stream)[0],
            M.unpermute(s["rows"], g, s["w"], s["base"], stream=stream)[0]]
    out += [*M.unpermute_backward(s["x"], g, s["w"], s["rows"], out=held(), stream=stream)]
    out += [M.unpermute_backward(s["x"], g, s["w"], out=held(), stream=stream)[0]]
    if s["x"].dtype == torch.bfloat16:
        live = int(g.offsets[-1])
        y, kept = M.unpermute(s["rows"], g, s["w"], s["base"], checkpoint=True, stream=stream)
        out += [y, kept[0][:live], kept[1][:live]]
        out += [*M.unpermute_backward(s["x"], g, s["w"], kept, out=held(), stream=stream)]
        codes = M.fp8_quantize_rows(s["x"])
        out += [M.permute(codes, g, out=held(), stream=stream)]
        q, qr = M.int8_quantize_rows(s["x"], stream=stream), M.int8_quantize_rows(s["rows"])
        w, u = M.int8_quantize_rows(s["we"], stream=stream), M.int8_quantize_rows(s["wu"])
        h = torch.bfloat16
        out += [*q, *w, M.int8_matmul(q, (w[0][0], w[1][0]), stream=stream),
                M.int8_matmul(q, (w[0][1], w[1][1]), w_up=(u[0][2], u[1][2]), stream=stream),
                M.int8_matmul(q, w, w_up=u, grouping=g, gather=True, out=held(h, 40), stream=stream),
                M.int8_matmul(qr, w, grouping=g, out=held(h, 40), stream=stream)]
    return out


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_same_results(M, dtype, monkeypatch):
    import torch
    from sigmoid_top_routing_router_amd import _lib
    s = state(M, dtype=getattr(torch, dtype))
    want = all_calls(M, s, torch.cuda.current_stream())

    class Counted:
        taken = 0

        def __getattr__(self, name):
            def f(*args):
                r = getattr(real, name)(*args)
                assert r is not None, name
                Counted.taken += 1
                return r
            return f
    real = _lib.calls
    monkeypatch.setattr(_lib, "calls", Counted())
    got = all_calls(M, s)
    assert Counted.taken == (18 if dtype == "bfloat16" else 7)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous()
        assert torch.equal(a, b)


def test_outputs_are_the_callers(M):
    import torch
    s = state(M)
    g = M.group_tokens(s["ids"], s["E"])
    out = torch.empty_like(s["rows"])
    assert M.permute(s["x"], g, out=out) is out
    assert M.unpermute_backward(s["x"], g, out=out)[0] is out
    w = M.int8_quantize_rows(s["we"])
    q, y = M.int8_quantize_rows(s["rows"]), torch.empty(len(out), 40, dtype=torch.int16, device="cuda")
    assert M.int8_matmul(q, w, grouping=g, out=y) is y
    # the grouping's parts do not overlap, and outlive each other
    parts = [g.counts, g.offsets, g.sorted_src, g.src_pos]
    copies = [p.clone() for p in parts]
    for i in range(4):
        parts[i].add_(1)
        copies[i].add_(1)
        for p, c in zip(parts, copies):
            assert torch.equal(p, c)
    keep = g.src_pos
    del g, parts
    torch.cuda.empty_cache()
    torch.full((1 << 20,), -5, device="cuda")
    assert torch.equal(keep, copies[3])


def test_what_is_not_ordinary_is_answered_by_python(M):
    import torch
    s = state(M)
    g = M.group_tokens(s["ids"], s["E"])
    x, rows, w = s["x"], s["rows"], s["w"]
    wide = torch.zeros(len(x), 512, dtype=x.dtype, device="cuda")
    q, wq = M.int8_quantize_rows(x), M.int8_quantize_rows(s["we"])
    both = torch.cat([x, rows])
    bad = [
        (ValueError, lambda: M.permute(wide[:, :256], g)),
        (ValueError, lambda: M.permute(x[:-1], g)),
        (TypeError, lambda: M.permute(x.double(), g)),
        (TypeError, lambda: M.permute(x.cpu(), g)),
        (TypeError, lambda: M.permute(x, g, out=rows.float())),
        (ValueError, lambda: M.permute(x, g, out=rows[:-1])),
        (M.MoeError, lambda: M.permute(both[:len(x)], g, out=both[len(x) - 1:-1])),
        (M.MoeError, lambda: M.unpermute(rows[:, :64].contiguous(), g, checkpoint=True)),
        (ValueError, lambda: M.permute_backward(rows[1:], g)),
        (ValueError, lambda: M.unpermute(rows, g, weights=w[:, :2])),
        (TypeError, lambda: M.unpermute(rows, g, weights=w.double())),
        (TypeError, lambda: M.unpermute(rows, g, base=x.float())),
        (M.MoeError, lambda: M.unpermute(rows.float(), g, checkpoint=True)),
        (ValueError, lambda: M.unpermute_backward(x, g, rows=rows[:-1])),
        (TypeError, lambda: M.unpermute_backward(x, g, rows=(rows, w))),
        (M.MoeError, lambda: M.group_tokens(s["ids"], 385)),
        (ValueError, lambda: M.int8_matmul((q[0], q[1][:-1]), (wq[0][0], wq[1][0]))),
        (ValueError, lambda: M.int8_matmul(q, wq)),
        (ValueError, lambda: M.int8_matmul(q, (wq[0][0], wq[1][0]), gather=True)),
        (TypeError, lambda: M.permute((x, None), g)),
        (TypeError, lambda: M.unpermute_backward(x, g, rows=(rows, None))),
        (ValueError, lambda: M.int8_matmul(q, (wq[0][0], wq[1][0]), w_up=(None, None))),
        (ValueError, lambda: M.int8_matmul(M.int8_quantize_rows(rows), wq, gather=True, grouping=(
            M.Grouping(g.counts, g.offsets, None, g.src_pos.view(-1, 1))))),
        (ValueError, lambda: M.int8_matmul(q, wq, grouping=M.Grouping(
            g.counts, None, g.sorted_src, g.src_pos), gather=True)),
        (M.MoeError, lambda: M.int8_quantize_rows(x[:, :24].contiguous())),
        (M.MoeError, lambda: M.group_tokens(s["ids"].repeat(1, 3), 6)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_current_stream_and_graph(M):
    import torch
    s = state(M, N=300)
    want = all_calls(M, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_calls(M, s)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    g = M.group_tokens(s["ids"], s["E"])
    M.unpermute(M.permute(s["x"], g), g, s["w"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = M.group_tokens(s["ids"], s["E"])
        y = M.unpermute(M.permute(s["x"], g), g, s["w"], s["base"])[0]
    for i in range(3):
        s["ids"].copy_(torch.randint(-1, s["E"], s["ids"].shape, device="cuda", dtype=torch.int32))
        s["x"].normal_()
        e = M.group_tokens(s["ids"], s["E"])
        eager = M.unpermute(M.permute(s["x"], e), e, s["w"], s["base"])[0].clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(g.src_pos, e.src_pos), i


def test_threads(M):
    import torch
    states = [state(M, N=64 + i, seed=i) for i in range(4)]
    want = [all_calls(M, s) for s in states]
    torch.cuda.synchronize()
    wrong = []

    def work(s, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = all_calls(M, s)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    wrong.append(len(s["x"]))
    threads = [threading.Thread(target=work, args=p) for p in zip(states, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_inference_mode_and_gradients_off(M):
    import torch
    s = state(M)
    want = all_calls(M, s)
    with torch.inference_mode():
        got = all_calls(M, s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    s["x"].requires_grad_(True)
    g = M.group_tokens(s["ids"], s["E"])
    assert not M.permute(s["x"], g).requires_grad

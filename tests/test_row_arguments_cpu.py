"""Arguments of the row calls that the binding has to answer before the C entry sees
them, without a GPU: the tensors are the host's, so the check that they are a GPU's
is taken out, and where there is a GPU nothing is called."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="there is a GPU")


@pytest.fixture
def M(monkeypatch):
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    real = M._dev

    def dev(t, name, dtype=None, shape=None):
        if isinstance(t, torch.Tensor):
            assert t.is_contiguous()
            if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
                raise TypeError(name)
            if shape is not None and t.shape != tuple(shape):
                raise ValueError(name)
            return t
        return real(t, name, dtype, shape)
    monkeypatch.setattr(M, "_dev", dev)
    return M


def kept(n, d):
    return torch.zeros(n, d, dtype=torch.uint8), torch.zeros(n, d // 128)


@pytest.mark.parametrize("d", [1, 64, 127, 192])
def test_codes_of_rows_without_whole_groups(M, d):
    """Below 128 columns the scales are an empty tensor, whose address is 0: the C
    entry would read the codes as rows of 16 bits, twice as many bytes."""
    pos = torch.zeros(4, 2, dtype=torch.int32)
    g = M.Grouping(None, None, None, pos)
    dy = torch.zeros(4, d, dtype=torch.bfloat16)
    assert kept(4, 64)[1].data_ptr() == 0
    for call in (lambda: M.permute(kept(4, d), g),
                 lambda: M.unpermute_backward(dy, g, rows=kept(8, d))):
        with pytest.raises(M.MoeError, match="multiple of 128") as e:
            call()
        assert e.value.status == 2


def test_a_grouping_without_tensors_is_no_dense_product(M, monkeypatch):
    """The extension module takes None in the place of offsets and places for a dense
    product, so a grouping that holds neither may not reach it."""
    from sigmoid_top_routing_router_amd import _lib

    class Dense:
        def int8_matmul(self, *args):
            return "a dense product"
    monkeypatch.setattr(_lib, "calls", Dense())
    q, w = (torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)), \
        (torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    assert M.int8_matmul(q, w) == "a dense product"
    for g in (M.Grouping(None, None, None, None),
              M.Grouping(None, None, torch.zeros(4, dtype=torch.int32), None)):
        with pytest.raises(ValueError, match=r"expected \(E, cols, 32\)"):
            M.int8_matmul(q, w, grouping=g)
    w3 = (w[0].view(1, 8, 32), w[1].view(1, 8))
    with pytest.raises(ValueError, match=r"src_pos must be \[N, K\]"):
        M.int8_matmul(q, w3, grouping=M.Grouping(None, None, None, None))


def test_a_workspace_has_the_bytes_that_it_says(M):
    """An expanded tensor's size is not the memory behind its address."""
    N, d, E, K, h = 4, 64, 3, 2, 32
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
    x, logits, ids = z(N, d), z(N, E, t=torch.float32), z(N, K, t=torch.int32)
    W = M.ExpertWeights(w_router=z(E, d), w_gate=z(E, h, d), w_up=z(E, h, d), w_down=z(E, d, h))
    calls = {
        "eqb_bias": lambda ws: M.eqb_bias(logits, K, workspace=ws),
        "forward": lambda ws: M.forward(x, W, K, workspace=ws),
        "backward": lambda ws: M.backward(x, x, W, logits, ids, workspace=ws),
        "rms_norm_backward": lambda ws: M.rms_norm_backward(x, x, z(d), workspace=ws),
        "balance_loss": lambda ws: M.balance_loss(logits, ids, workspace=ws),
        "group_tokens": lambda ws: M.group_tokens(ids, E, workspace=ws),
    }
    small = torch.zeros(256, dtype=torch.uint8)
    for name, call in calls.items():
        for ws in (small[:1].expand(1 << 20), torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0]):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                call(ws)
                pytest.fail(name)

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

"""The binding's extension module without a GPU: on anything but ordinary arguments
it returns None, and the Python code answers with its own checks."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def M():
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def test_none_for_anything_else(M):
    from sigmoid_top_routing_router_amd import _lib
    c = _lib.calls
    rows, pos = torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    calls = {"group": 2, "permute": 4, "permute_backward": 2, "unpermute": 5,
             "unpermute_backward": 6, "int8_quantize_rows": 1, "int8_matmul": 10}
    for name, n in calls.items():
        f = getattr(c, name)
        for args in ([], [None] * n, [1] * n, [rows] * n, [pos] * n, [rows] * (n + 1), ["x"] * n,
                     [rows, pos] * n):
            assert f(*args) is None, (name, args)


def test_python_checks_answer(M):
    rows, pos = torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    g = M.Grouping(None, None, None, pos)
    for call in (lambda: M.group_tokens(pos, 3), lambda: M.permute(rows, g),
                 lambda: M.permute_backward(rows, g), lambda: M.unpermute(rows, g),
                 lambda: M.unpermute_backward(rows, g), lambda: M.int8_quantize_rows(rows),
                 lambda: M.int8_matmul((rows, rows), (rows, rows))):
        with pytest.raises(TypeError, match="GPU torch tensor"):
            call()


def test_bind_refuses(M):
    from sigmoid_top_routing_router_amd import _lib
    with pytest.raises(TypeError):
        _lib.calls.bind(1)
    with pytest.raises(ValueError):
        _lib.calls.bind(*[0] * 8)
    with pytest.raises(TypeError):
        _lib.calls.bind(*["x"] * 8)


def test_without_the_module(M, monkeypatch):
    """A module that does not load leaves the way through Python, and says so."""
    import sys
    from sigmoid_top_routing_router_amd import _lib
    monkeypatch.setitem(sys.modules, "sigmoid_top_routing_router_amd._calls", None)
    monkeypatch.delattr(M, "_calls", raising=False)
    with pytest.warns(UserWarning, match="twice the time"):
        calls = _lib._bind_calls(M.load_library())
    assert calls.permute(1, 2, 3, 4) is None
    monkeypatch.setattr(_lib, "calls", calls)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError, match="GPU torch tensor"):
        M.group_tokens(pos, 3)

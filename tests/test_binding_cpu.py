"""The binding's extension module is used only beside the torch, the Python and the C
library that it was built with."""
import warnings

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_router_amd import _lib
    return _lib.load()


def is_short(calls):
    return type(calls).__name__ == "module"


def test_built_for_this_torch(lib):
    from sigmoid_top_routing_router_amd import _lib
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        calls = _lib._bind_calls(lib)
    assert is_short(calls)
    assert torch.__version__ in calls.built_for and torch.version.git_version in calls.built_for
    assert calls.abi_version == lib.moe_abi_version()


def test_another_torch_loads_but_is_not_used(lib, monkeypatch):
    from sigmoid_top_routing_router_amd import _lib
    monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    with pytest.warns(UserWarning, match="another torch.*here is torch .* 0000"):
        calls = _lib._bind_calls(lib)
    assert not is_short(calls) and calls.permute(1, 2, 3, 4) is None


def test_a_module_without_a_stamp_is_not_used(lib, monkeypatch):
    from sigmoid_top_routing_router_amd import _calls, _lib
    monkeypatch.delattr(_calls, "built_for")
    with pytest.warns(UserWarning, match="twice the time"):
        assert not is_short(_lib._bind_calls(lib))


def test_another_library_is_not_called(lib, monkeypatch):
    from sigmoid_top_routing_router_amd import _lib

    class Other:
        def __getattr__(self, name):
            return getattr(lib, name)

        def moe_abi_version(self):
            return lib.moe_abi_version() + 1
    with pytest.warns(UserWarning, match="of ABI"):
        assert not is_short(_lib._bind_calls(Other()))


def test_library_without_the_module(tmp_path, monkeypatch):
    """Where the module does not build, the library does, and no older module stays."""
    import ctypes
    import os
    import shutil

    from sigmoid_top_routing_router_amd import build as B
    if not os.path.exists("/opt/rocm/bin/hipcc") and shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    src = tmp_path / "one.cpp"
    src.write_text('extern "C" int one() { return 1; }\n')
    older = tmp_path / "_calls.so"
    older.write_text("")

    def no_headers(verbose=False):
        raise RuntimeError("Python.h: no such file")
    monkeypatch.setattr(B, "sources", lambda: [str(src)])
    monkeypatch.setattr(B, "OBJ", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "BINDING", str(older))
    monkeypatch.setattr(B, "build_binding", no_headers)
    monkeypatch.setattr(B, "build_probes", lambda verbose=False: [])
    with pytest.warns(UserWarning, match="Python.h: no such file"):
        lib = B.build()
    assert ctypes.CDLL(lib).one() == 1 and not older.exists()

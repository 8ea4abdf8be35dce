"""Refusals of the entry points around the layer, each from a call that is
valid but for the one argument under test: the message says that this argument
was the reason.

The addresses are a host buffer's.  On a host without a GPU the valid call
passes every check and ends at its first launch (MOE_ERR_HIP); where there is
a GPU the calls are not made, a missing check would launch on those addresses."""
import ctypes as C
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sigmoid_top_routing_router_amd", "libmoe_mi355x.so")
pytestmark = [pytest.mark.skipif(not os.path.exists(LIB), reason="library not built"),
              pytest.mark.skipif(torch.cuda.device_count() > 0, reason="there is a GPU")]

PAGE = 1 << 16  # every buffer of the calls below fits one
OK_TO_LAUNCH = 4


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_router_amd import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def page():
    """page(i): the address of the i-th of 40 pages, 256-byte aligned."""
    buf = C.create_string_buffer(40 * PAGE + 256)
    base = (C.cast(buf, C.c_void_p).value + 255) // 256 * 256
    yield lambda i: base + i * PAGE
    del buf


def refused(lib, status, words):
    return status == 1 and words in lib.moe_last_error_message().decode()


# ---------------------------------------------------------------- layer backward
WEIGHTS = ["w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"]


def backward_call(lib, page):
    """A function that makes the call with some arguments changed, and the
    addresses it uses by name."""
    from sigmoid_top_routing_router_amd._lib import MoeGrads, MoeProblem, MoeWeights
    p = MoeProblem(N=4, d=64, E=4, K=2, h=32, n_shared=1, h_shared=32, flags=0)
    names = ["x", "dy", "z", "ids", "gz", *WEIGHTS, "g.x", "g.logits", *["g." + w for w in WEIGHTS]]
    at = {n: page(i) for i, n in enumerate(names)}
    at["ws"] = page(len(names))
    need = lib.moe_backward_workspace_bytes(C.byref(p))
    assert 0 < need <= (40 - len(names)) * PAGE

    def call(wsb=need, flags=0, **kw):
        a = {**at, **{k.replace("g_", "g."): v for k, v in kw.items()}}
        p.flags = flags
        w = MoeWeights(*[a[k] for k in WEIGHTS])
        g = MoeGrads(a["g.x"], a["g.logits"], *[a["g." + k] for k in WEIGHTS])
        return lib.moe_backward(C.byref(p), C.byref(w), a["x"], a["dy"], a["z"], a["ids"], a["gz"],
                                C.byref(g), a["ws"], wsb, None)
    return call, at


def test_backward_aliases(lib, page):
    call, at = backward_call(lib, page)
    assert call() == OK_TO_LAUNCH
    assert call(gz=None) == OK_TO_LAUNCH
    assert call(g_logits=at["gz"]) == OK_TO_LAUNCH            # in place
    inputs = ["x", "dy", "z", "ids", *WEIGHTS]
    outputs = ["g_x", "g_logits", *["g_" + w for w in WEIGHTS]]
    for o in outputs:
        for i in inputs:
            assert refused(lib, call(**{o: at[i]}), "aliases an input"), (o, i)
        if o != "g_logits":
            assert refused(lib, call(**{o: at["gz"]}), "aliases an input"), o
        for q in outputs:
            if q != o:
                status = call(**{o: at[q.replace("g_", "g.")]})
                assert refused(lib, status, "two outputs"), (o, q)
    # a part of a buffer is enough: grad_x is 512 bytes, the logits 64
    assert refused(lib, call(g_x=at["x"] + 496), "aliases an input")
    assert call(g_x=at["x"] + 512) == OK_TO_LAUNCH
    assert refused(lib, call(g_logits=at["gz"] + 32), "aliases an input")
    assert refused(lib, call(g_logits=at["g.x"] + 256), "two outputs")
    assert refused(lib, call(ws=at["dy"] + 256), "aliases an input")
    assert refused(lib, call(ws=at["g.w_down"]), "two outputs")


def test_backward_refusals_name_their_reason(lib, page):
    """Every requirement of the header, one at a time."""
    call, at = backward_call(lib, page)
    assert call() == OK_TO_LAUNCH
    for n in ("x", "dy", "z", "ids"):
        assert refused(lib, call(**{n: None}), "are required"), n
    for n in ("w_gate", "w_up", "w_down", "g_x", "g_logits", "g_w_gate", "g_w_up", "g_w_down"):
        assert refused(lib, call(**{n: None}), "routed expert weights and the gradients"), n
    for n in ("ws_gate", "ws_up", "ws_down"):
        assert refused(lib, call(**{n: None}), "shared expert weights"), n
        assert refused(lib, call(**{"g_" + n: None}), "shared expert weights"), n
    assert refused(lib, call(w_router=None), "both or neither")
    assert refused(lib, call(g_w_router=None), "both or neither")
    assert call(w_router=None, g_w_router=None) == OK_TO_LAUNCH
    for n in ("x", "dy", *WEIGHTS):
        assert refused(lib, call(**{n: at[n] + 8}), "bf16 inputs must be 16-byte aligned"), n
    for n in ("x", *WEIGHTS):
        status = call(**{"g_" + n: at["g." + n] + 8})
        assert refused(lib, status, "bf16 gradients must be 16-byte aligned"), n
    for n in ("z", "ids", "gz"):
        assert refused(lib, call(**{n: at[n] + 2}), "logits and ids must be 4-byte aligned"), n
    assert refused(lib, call(g_logits=at["g.logits"] + 2), "logits and ids must be 4-byte")
    assert refused(lib, call(flags=4), "row-major weights only")
    assert refused(lib, call(flags=16), "unknown flag bits")
    assert call(flags=11) == OK_TO_LAUNCH                     # the forward call's routing flags
    assert refused(lib, call(ws=None), "workspace must be non-NULL and 256-byte aligned")
    assert refused(lib, call(ws=at["ws"] + 4), "workspace must be non-NULL and 256-byte aligned")
    assert call(wsb=64) == 3


# ---------------------------------------------------------------- balance loss
def balance_calls(lib, page):
    names = ["z", "ids", "cin", "b", "e", "loss", "cout", "mean", "gl", "gin", "out", "ws"]
    at = {n: page(i) for i, n in enumerate(names)}
    need = lib.moe_balance_workspace_bytes(40, 8, 3)
    assert 0 < need <= PAGE

    def forward(wsb=need, **kw):
        a = dict(at, N=40, E=8, K=2, G=3, score=1, coef=1e-2, wsb=wsb, **{})
        a.update(kw)
        return lib.moe_balance_loss(*[a[k] for k in (
            "z", "ids", "cin", "b", "e", "N", "E", "K", "G", "score", "coef", "loss", "cout",
            "mean", "ws", "wsb")], None)

    def backward(**kw):
        a = dict(at, N=40, E=8, G=3, score=1, coef=1e-2)
        a.update(kw)
        return lib.moe_balance_loss_backward(*[a[k] for k in (
            "z", "cin", "b", "e", "N", "E", "G", "score", "coef", "gl", "gin", "out")], None)
    return forward, backward, at


def test_balance_aliases(lib, page):
    forward, backward, at = balance_calls(lib, page)
    assert forward() == OK_TO_LAUNCH and backward() == OK_TO_LAUNCH
    for o in ("loss", "cout", "mean", "ws"):
        for i in ("z", "ids", "cin", "b", "e"):
            assert refused(lib, forward(**{o: at[i]}), "aliases an input"), (o, i)
        for q in ("loss", "cout", "mean", "ws"):
            if q != o and "ws" not in (o, q):
                assert refused(lib, forward(**{o: at[q]}), "two outputs"), (o, q)
    assert refused(lib, forward(mean=at["cout"] + 92), "two outputs")     # 96 bytes each
    assert forward(mean=at["cout"] + 96) == OK_TO_LAUNCH
    assert refused(lib, forward(loss=at["ws"] + 4), "two outputs")
    assert backward(out=at["gin"]) == OK_TO_LAUNCH                        # in place
    for i in ("z", "cin", "b", "e", "gl"):
        assert refused(lib, backward(out=at[i]), "aliases an input"), i
    assert refused(lib, backward(out=at["gin"] + 32), "aliases an input")
    assert refused(lib, backward(gl=at["out"] + 128), "aliases an input")


# ---------------------------------------------------------------- norm
def norm_calls(lib, page):
    names = ["x", "res", "w", "post", "y", "r", "codes", "scales", "dy", "dres", "dx", "dr", "dw",
             "dp", "ws"]
    at = {n: page(i) for i, n in enumerate(names)}
    need = lib.moe_rms_norm_backward_workspace_bytes(4, 128)
    assert 0 < need <= PAGE
    size = dict(n=4, d=128, eps=1e-6, flags=0, wsb=need)

    def forward(**kw):
        a = {**at, **size, **kw}
        return lib.moe_rms_norm(*[a[k] for k in (
            "x", "res", "post", "w", "n", "d", "eps", "flags", "y", "r", "codes", "scales")], None)

    def backward(**kw):
        a = {**at, "r": at["res"], **size, **kw}
        return lib.moe_rms_norm_backward(*[a[k] for k in (
            "dy", "r", "x", "dres", "w", "post", "n", "d", "eps", "flags", "dx", "dr", "dw", "dp",
            "ws", "wsb")], None)
    return forward, backward, at


def test_norm_aliases(lib, page):
    forward, backward, at = norm_calls(lib, page)
    assert forward() == OK_TO_LAUNCH and backward() == OK_TO_LAUNCH
    assert forward(r=at["res"]) == OK_TO_LAUNCH                           # in place
    for o in ("y", "r", "codes", "scales"):
        for i in ("x", "res", "w", "post"):
            if (o, i) != ("r", "res"):
                assert refused(lib, forward(**{o: at[i]}), "aliases an input"), (o, i)
        for q in ("y", "r", "codes", "scales"):
            if q != o:
                assert refused(lib, forward(**{o: at[q]}), "two outputs"), (o, q)
    assert refused(lib, forward(r=at["res"] + 256), "aliases an input")   # the next row
    assert refused(lib, forward(y=at["r"] + 768), "two outputs")
    for o in ("dx", "dr", "dw", "dp", "ws"):
        for i in ("dy", "res", "x", "dres", "w", "post"):
            assert refused(lib, backward(**{o: at[i]}), "aliases an input"), (o, i)
        for q in ("dx", "dr", "dw", "dp"):
            if q != o:
                assert refused(lib, backward(**{o: at[q]}), "two outputs"), (o, q)
    assert refused(lib, backward(dr=at["dx"] + 256), "two outputs")


def test_norm_backward_of_no_rows(lib, page):
    """n = 0: with weight gradients they are zeros (a launch), without there is
    nothing to write; an empty tensor's address is NULL."""
    _, backward, at = norm_calls(lib, page)
    rows = {k: None for k in ("dy", "r", "x", "dres", "dx", "dr")}
    assert backward(n=0, **rows, dw=None, dp=None) == 0
    assert backward(n=0, **rows, dw=None, dp=None, post=None) == 0
    assert backward(n=0, dw=None, dp=None, post=None, x=None) == 0
    assert backward(n=0, **rows) == OK_TO_LAUNCH
    assert backward(n=0, **rows, dp=None) == OK_TO_LAUNCH
    # what is refused for rows is refused without them
    assert refused(lib, backward(n=0, **rows, dw=None, dp=None, w=None), "weight is required")
    assert refused(lib, backward(n=0, **rows, dw=None, post=None), "needs post_weight")
    assert refused(lib, backward(n=0, **rows, dw=None, dp=None, eps=-1.0), "eps")
    assert refused(lib, backward(dx=None, dr=None, dw=None, dp=None), "an output is required")

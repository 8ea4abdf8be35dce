"""Refusals of the entry points that take the layer apart, each from a call that
is valid but for the one argument under test: the message says that this
argument was the reason.

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

PAGE = 1 << 16
INVALID, SHAPE, SMALL, LAUNCH = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_router_amd import _lib
    return _lib.load()


@pytest.fixture(scope="module")
def page():
    buf = C.create_string_buffer(20 * PAGE + 256)
    base = (C.cast(buf, C.c_void_p).value + 255) // 256 * 256
    yield lambda i: base + i * PAGE
    del buf


def says(lib, got, status, words):
    return got == status and words in lib.moe_last_error_message().decode()


def maker(lib, page, fn, names, defaults):
    """call(**changes) with a page for every buffer of names."""
    at = {n: page(i) for i, n in enumerate(names)}

    def call(**kw):
        return fn(lib, {**at, **defaults, **kw})
    return call, at


def check_aliases(lib, call, at, inputs, outputs):
    for o in outputs:
        for i in inputs:
            assert says(lib, call(**{o: at[i]}), INVALID, "aliases an input"), (o, i)
            # the last byte of the input is enough
        for q in outputs:
            if q != o:
                assert says(lib, call(**{o: at[q]}), INVALID, "two outputs"), (o, q)


def test_group(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_group(
        a["ids"], a["N"], a["E"], a["K"], a["counts"], a["offsets"], a["src"], a["pos"], a["ws"],
        a["wsb"], None), ["ids", "counts", "offsets", "src", "pos", "ws"],
        dict(N=4, E=3, K=2, wsb=PAGE))
    assert call() == LAUNCH
    assert call(N=0, ids=None, src=None, pos=None) == LAUNCH     # zeros leave all the same
    assert call(K=8, E=1) == LAUNCH
    check_aliases(lib, call, at, ["ids"], ["counts", "offsets", "src", "pos"])
    assert says(lib, call(ws=at["ids"]), INVALID, "aliases an input")
    assert says(lib, call(ws=at["pos"]), INVALID, "two outputs")
    for n in ("ids", "src", "pos"):
        assert says(lib, call(**{n: None}), INVALID, "topk_ids, sorted_src and src_pos"), n
    for n in ("counts", "offsets"):
        assert says(lib, call(**{n: None}), INVALID, "counts and offsets are required"), n
    for n in ("ids", "counts", "offsets", "src", "pos"):
        assert says(lib, call(**{n: at[n] + 2}), INVALID, "4-byte aligned"), n
    for kw in (dict(N=-1), dict(N=(1 << 24) + 1), dict(E=0), dict(E=385), dict(K=0), dict(K=9)):
        assert says(lib, call(**kw), SHAPE, "need 0 <= N"), kw
        assert lib.moe_group_workspace_bytes(kw.get("N", 4), kw.get("E", 3), kw.get("K", 2)) == 0
    assert says(lib, call(ws=None), INVALID, "256-byte aligned")
    assert says(lib, call(ws=at["ws"] + 16), INVALID, "256-byte aligned")
    assert says(lib, call(wsb=8), SMALL, "workspace")


ROWS = dict(N=4, d=256, K=2, flags=0)


def check_sizes(lib, call):
    for kw in (dict(N=-1), dict(N=(1 << 24) + 1), dict(d=0), dict(d=8193), dict(K=0), dict(K=9)):
        assert says(lib, call(**kw), SHAPE, "need 0 <= N"), kw
    assert says(lib, call(flags=2), INVALID, "unknown flag bits")
    assert call(N=0) == 0


def test_permute(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_permute(
        a["x"], a["xs"], a["pos"], a["N"], a["d"], a["K"], a["flags"], a["rows"], None),
        ["x", "xs", "pos", "rows"], ROWS)
    assert call() == LAUNCH and call(xs=None) == LAUNCH and call(xs=None, flags=1) == LAUNCH
    assert call(xs=None, d=77, x=at["x"] + 2, rows=at["rows"] + 2) == LAUNCH
    check_sizes(lib, lambda **kw: call(**{"xs": None, **kw}))
    check_aliases(lib, call, at, ["x", "xs", "pos"], ["rows"])
    for n in ("x", "pos", "rows"):
        assert says(lib, call(**{n: None}), INVALID, "x, src_pos and rows are required"), n
    assert says(lib, call(flags=1), INVALID, "belong to bf16 rows")
    assert says(lib, call(d=192), SHAPE, "multiple of 128")
    for n in ("x", "rows"):
        assert says(lib, call(**{n: at[n] + 8}), INVALID, "16-byte aligned"), n
        assert says(lib, call(xs=None, **{n: at[n] + 1}), INVALID, "2-byte aligned"), n
        assert says(lib, call(xs=None, flags=1, **{n: at[n] + 2}), INVALID, "4-byte aligned"), n
    for n in ("xs", "pos"):
        assert says(lib, call(**{n: at[n] + 2}), INVALID, "4-byte aligned"), n


def test_permute_backward(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_permute_backward(
        a["g"], a["pos"], a["N"], a["d"], a["K"], a["flags"], a["dx"], None), ["g", "pos", "dx"],
        ROWS)
    assert call() == LAUNCH and call(flags=1) == LAUNCH
    check_sizes(lib, call)
    check_aliases(lib, call, at, ["g", "pos"], ["dx"])
    for n in ("g", "pos", "dx"):
        assert says(lib, call(**{n: None}), INVALID, "grad_rows, src_pos and grad_x"), n
    for n in ("g", "dx"):
        assert says(lib, call(**{n: at[n] + 1}), INVALID, "2-byte aligned"), n
    assert says(lib, call(pos=at["pos"] + 2), INVALID, "4-byte aligned")


def test_unpermute(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_unpermute(
        a["rows"], a["pos"], a["w"], a["base"], a["N"], a["d"], a["K"], a["flags"], a["y"],
        a["codes"], a["scales"], None), ["rows", "pos", "w", "base", "y", "codes", "scales"], ROWS)
    plain = dict(codes=None, scales=None)
    assert call() == LAUNCH and call(**plain) == LAUNCH and call(w=None, base=None) == LAUNCH
    assert call(flags=1, **plain) == LAUNCH and call(d=77, **plain) == LAUNCH
    check_sizes(lib, lambda **kw: call(**{**plain, **kw}))
    check_aliases(lib, call, at, ["rows", "pos", "w", "base"], ["y", "codes", "scales"])
    assert says(lib, call(codes=None), INVALID, "both or neither")
    assert says(lib, call(scales=None), INVALID, "both or neither")
    for n in ("rows", "pos", "y"):
        assert says(lib, call(**{n: None}), INVALID, "rows, src_pos and y are required"), n
    assert says(lib, call(flags=1), INVALID, "belong to bf16 rows")
    assert says(lib, call(d=192), SHAPE, "multiple of 128")
    for n in ("rows", "base", "y", "codes"):
        assert says(lib, call(**{n: at[n] + 8}), INVALID, "16-byte aligned"), n
    for n in ("rows", "base", "y"):
        assert says(lib, call(**plain, **{n: at[n] + 1}), INVALID, "2-byte aligned"), n
    for n in ("pos", "w", "scales"):
        assert says(lib, call(**{n: at[n] + 2}), INVALID, "4-byte aligned"), n


def test_unpermute_backward(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_unpermute_backward(
        a["dy"], a["rows"], a["rs"], a["pos"], a["w"], a["N"], a["d"], a["K"], a["flags"],
        a["dr"], a["dw"], None), ["dy", "rows", "rs", "pos", "w", "dr", "dw"], ROWS)
    assert call() == LAUNCH and call(rs=None) == LAUNCH and call(rs=None, flags=1) == LAUNCH
    assert call(dr=None) == LAUNCH and call(dw=None, rows=None, rs=None) == LAUNCH
    assert call(w=None) == LAUNCH
    check_sizes(lib, lambda **kw: call(**{"rs": None, **kw}))
    check_aliases(lib, call, at, ["dy", "rows", "rs", "pos", "w"], ["dr", "dw"])
    assert says(lib, call(dr=None, dw=None), INVALID, "grad_rows or grad_weights is required")
    for n in ("dy", "pos"):
        assert says(lib, call(**{n: None}), INVALID, "grad_y and src_pos are required"), n
    assert says(lib, call(rows=None), INVALID, "grad_weights needs rows")
    assert says(lib, call(flags=1), INVALID, "belong to bf16 rows")
    assert says(lib, call(d=192), SHAPE, "multiple of 128")
    for n in ("dy", "rows", "dr"):
        assert says(lib, call(**{n: at[n] + 8}), INVALID, "16-byte aligned"), n
    for n in ("pos", "w", "rs", "dw"):
        assert says(lib, call(**{n: at[n] + 2}), INVALID, "4-byte aligned"), n


def test_int8_quantize_rows(lib, page):
    call, at = maker(lib, page, lambda l, a: l.moe_int8_quantize_rows(
        a["x"], a["n"], a["c"], a["q"], a["s"], None), ["x", "q", "s"], dict(n=3, c=48))
    assert call() == LAUNCH and call(n=0, x=None) == 0
    check_aliases(lib, call, at, ["x"], ["q", "s"])
    for kw in (dict(n=-1), dict(n=(1 << 27) + 1), dict(c=0), dict(c=8), dict(c=56),
               dict(c=65552)):
        assert says(lib, call(**kw), SHAPE, "cols % 16 == 0"), kw
    for n in ("x", "q", "s"):
        assert says(lib, call(**{n: None}), INVALID, "are required"), n
    for n in ("x", "q"):
        assert says(lib, call(**{n: at[n] + 8}), INVALID, "16-byte aligned"), n
    assert says(lib, call(s=at["s"] + 2), INVALID, "4-byte aligned")


def test_int8_matmul(lib, page):
    from sigmoid_top_routing_router_amd._lib import MoeInt8Matmul
    names = ["a", "sa", "w", "sw", "u", "su", "off", "src", "out"]

    def fn(l, a):
        p = MoeInt8Matmul(a["ar"], a["r"], a["k"], a["cols"], a["E"], a["K"],
                          *[a[n] for n in names[:-1]])
        return l.moe_int8_matmul(C.byref(p), a["out"], None)
    call, at = maker(lib, page, fn, names, dict(ar=4, r=8, k=48, cols=24, E=3, K=2))
    assert call() == LAUNCH and call(u=None, su=None) == LAUNCH
    assert call(src=None, ar=8) == LAUNCH
    assert call(off=None, src=None, E=1, ar=8) == LAUNCH
    assert call(r=0) == 0
    check_aliases(lib, call, at, names[:-1], ["out"])
    for kw in (dict(r=-1), dict(r=(1 << 27) + 1), dict(ar=-1), dict(ar=(1 << 27) + 1), dict(k=0),
               dict(k=40), dict(k=65552), dict(cols=0), dict(cols=20), dict(cols=65544),
               dict(E=0), dict(E=385), dict(K=0), dict(K=9)):
        assert says(lib, call(**kw), SHAPE, "k % 16 == 0"), kw
    assert says(lib, call(ar=65536, k=65536), SHAPE, "a gathered a")
    assert says(lib, call(off=None), INVALID, "one weight and no sorted_src")
    assert says(lib, call(off=None, src=None), INVALID, "one weight and no sorted_src")
    assert says(lib, call(off=None, E=1), INVALID, "one weight and no sorted_src")
    assert says(lib, call(u=None), INVALID, "both or neither")
    assert says(lib, call(su=None), INVALID, "both or neither")
    assert says(lib, call(src=None), INVALID, "a_rows must be rows")
    assert says(lib, call(ar=0), INVALID, "rows of an empty a")
    for n in ("a", "sa", "w", "sw", "out"):
        assert says(lib, call(**{n: None}), INVALID, "are required"), n
    for n in ("a", "w", "u", "out"):
        assert says(lib, call(**{n: at[n] + 8}), INVALID, "16-byte aligned"), n
    for n in ("sa", "sw", "su", "off", "src"):
        assert says(lib, call(**{n: at[n] + 2}), INVALID, "4-byte aligned"), n
    assert says(lib, lib.moe_int8_matmul(None, at["out"], None), INVALID, "problem is NULL")


def test_struct_layout_matches_header(tmp_path):
    import shutil
    import subprocess
    from sigmoid_top_routing_router_amd._lib import MoeInt8Matmul
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    prog = tmp_path / "layout.c"
    header = os.path.join(ROOT, "include", "moe_mi355x.h")
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{header}"',
             'int main(void){printf("%zu", sizeof(moe_int8_matmul_t));']
    lines += [f'printf(" %zu", offsetof(moe_int8_matmul_t, {f}));' for f, _ in MoeInt8Matmul._fields_]
    prog.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run([cc, str(prog), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [C.sizeof(MoeInt8Matmul)] + \
        [getattr(MoeInt8Matmul, f).offset for f, _ in MoeInt8Matmul._fields_]

"""The loads into LDS that the layer's backward pass issues in assembly carry
their own wait states: a vector-memory read of a scalar register needs five of
them after a vector instruction that wrote it (v_readfirstlane makes the
descriptors and the offsets), and one after m0 was written.  The compiler counts
them for its own instructions only, not for what stands inside an asm block."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "sigmoid_top_routing_router_amd", "csrc", "layer_grad.hip")


def strings(text, macros):
    """The string literals of a piece of source, macros opened, one after the
    other."""
    out = ""
    for lit, name, args in re.findall(r'"((?:[^"\\]|\\.)*)"|(MOE_DMA\w*)(?:\(([^)]*)\))?', text):
        out += strings(macros[name], {}) + args if name else lit
    return out.replace("\\n", "\n").replace("\\t", "\t")


def blocks():
    src = open(SOURCE).read()
    macros = dict(re.findall(r"#define (MOE_DMA\w*)(?:\([^)]*\))? (.*)", src))
    for body in re.findall(r"asm volatile\((.*?)::", src, re.S):
        code = strings(body, macros)
        if "buffer_load" in code:
            yield [line.strip() for line in code.replace('"', "\n").split("\n") if line.strip()]


def test_wait_states_of_the_loads():
    seen = 0
    for code in blocks():
        seen += 1
        states, since_m0 = 0, None
        loads = 0
        for line in code:
            op = re.match(r"[a-z_0-9]+", line)
            op = op.group(0) if op else ""
            if op.startswith("buffer_load"):
                if loads == 0:
                    assert states >= 5, code       # behind whatever stood in front of the block
                assert since_m0 is not None and since_m0 >= 1, code
                loads += 1
            if op:
                n = int(line.split()[1]) + 1 if op == "s_nop" else 1
                states += n
                if since_m0 is not None:
                    since_m0 += n
                if op.startswith("s_") and " m0," in line:
                    since_m0 = 0
        assert loads >= 1, code
    assert seen == 3

"""Which kernels of the linear layer the bounds-checking build checks, read from the source: each kernel that
addresses the workspace or a tensor directly (not through TMA, which clips) guards those accesses."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "output_head_kl_b200", "csrc")


def _function(source, name):
    """The text of a function from its name to the closing brace of its body."""
    at = source.index(name + "(")
    start = at + re.search(r"\)\s*(const\s*)?\{", source[at:]).end()
    depth, i = 1, start
    while depth:
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        i += 1
    return source[at:i]


def _checks(text):
    return re.findall(r"dbg_ok\((.*?), (?:p\.)?flags\)", text, re.S)


def test_linear_kernels_check_what_tma_does_not_clip():
    with open(os.path.join(CSRC, "linear.cu")) as f:
        source = f.read()
    pair = _checks(_function(source, "linear_pair_kernel"))
    assert any("p.part_floats" in c and "kMaxSplitTiles" in c for c in pair)         # share and ticket
    small = _checks(_function(source, "linear_small_kernel"))
    assert sum("row < p.M" in c and "p.N" in c for c in small) == 2                  # side data, outputs
    slopes = _checks(_function(source, "act_grad_kernel"))
    assert any("r1 <= M" in c for c in slopes) and any("part_floats" in c for c in slopes)
    assert any("p.N" in c for c in _checks(_function(source, "void load_side")))
    assert len(_checks(_function(source, "void store32"))) == 1 and len(_checks(_function(source, "void load_res"))) == 1


def test_the_exception_is_documented():
    """norm.cu holds no checks (its calls have no flag word), and the header says so."""
    with open(os.path.join(CSRC, "norm.cu")) as f:
        assert "dbg_ok" not in f.read()
    with open(os.path.join(CSRC, "..", "..", "include", "kdkl.h")) as f:
        assert "the RMS norm's kernels have no flag word and no such checks" in f.read()

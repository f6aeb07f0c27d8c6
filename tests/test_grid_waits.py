"""A kernel that may start before the launch in front of it has ended reads nothing in front of its
wait (CPU: reads the sources).

What the launches in front have written is only promised to the grid that waits, behind its wait,
whatever the launch in front has itself waited for: queries, lengths and pages of a call may have
been written by the launch before the call's first.  A kernel that runs beside the one in front may
read them where that one passes on what it has seen, by a word that it releases and this one
acquires; then by coherent loads alone.
"""
import os
import re

import pytest

from speculative_decode_verify_sdv_gb300 import build

FILES = ["page_assign.cu", "qk_norm_rope.cu", "prefix_attn.cu", "prefix_own.cu", "prefix_tc_kernel.cuh",
         "verify_drafts.cu", "paged_attn.cu", "attn_tc_kernel.cuh",
         "linear_attn.cu", "linear_tc_kernel.cuh", "linear_window.cu"]
READS = (r"\b(?:__ldg|__ldcg|tma_load\w*|attn_seq|attn_word|lin_tokens|prefix_length|page_need|place_row|"
         r"griddep_launch_dependents)\s*\(|\.start\(|<const (?:u?int\d|float\d|uint)\w*\s*\*>\(a\.")


def kernels(text):
    """Name and body of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        name = re.compile(r"\b(\w+)\s*\(").search(text, m.end())
        if name.group(1) == "__launch_bounds__":
            name = re.compile(r"\b(\w+)\s*\(").search(text, _closing(text, name.end() - 1, "(", ")"))
        at = text.index("{", _closing(text, name.end() - 1, "(", ")"))
        yield name.group(1), text[at + 1:_closing(text, at, "{", "}")]


def _closing(text, at, opening, closing):
    depth = 0
    for i in range(at, len(text)):
        depth += {opening: 1, closing: -1}.get(text[i], 0)
        if depth == 0:
            return i
    raise AssertionError("not closed")


def early_reads(body):
    """What a body reads (or starts) before it waits unconditionally; None where it never does."""
    for m in re.finditer(r"griddep_wait\(\);", body):
        front = body[:m.start()]
        if front.count("{") != front.count("}"):
            continue
        if front.rstrip()[-1:] in ("", ";", "}", "{"):
            return re.findall(READS, front)
        guard = re.search(r"if \(!(\w+)\)\s*$", front)
        if guard and re.search(rf"\b{guard.group(1)} = [^;]*\bpassed_on\(", front):
            return re.findall(READS, front) + re.findall(r"\b(?:__ldg|attn_word)\(", body[m.end():])
    return None


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_in_front_of_the_wait(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = dict(kernels(text))
    assert found
    assert {k: early_reads(body) for k, body in found.items()} == {k: [] for k in found}


def test_a_late_or_conditional_wait_is_found():
    text = "__global__ void __launch_bounds__(f(1), 2) k(const A a) { int x = __ldg(a.p); griddep_wait(); }"
    assert [(n, early_reads(b)) for n, b in kernels(text)] == [("k", ["__ldg("])]
    assert early_reads("if (x) griddep_wait(); y = 1;") is None
    assert early_reads("if (x) { griddep_wait(); }") is None
    assert early_reads("x = passed_on(w); if (!x) griddep_wait(); y = __ldcg(p);") == []
    assert early_reads("x = passed_on(w); if (!x) griddep_wait(); y = __ldg(p);") == ["__ldg("]
    assert early_reads("x = 1; if (!x) griddep_wait(); y = __ldcg(p);") is None
    assert early_reads("if (x) { y = 1; } griddep_wait(); z = __ldg(p);") == []

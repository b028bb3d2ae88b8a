"""Checks of the kernels' sources for mistakes that a run shows only by chance (no GPU needed)."""
import os
import re

import pytest

from deepseek_sparse_attention_lightning_gb300 import build


def _code(name):
    """A source file without its comments."""
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)


def _enclosing_calls(text, at):
    """Names of the calls whose parentheses enclose position `at`, within its statement."""
    names, depth = [], 0
    for i in range(at - 1, -1, -1):
        c = text[i]
        if c in ";{}" and depth == 0:
            break
        if c == ")":
            depth += 1
        elif c == "(":
            if depth:
                depth -= 1
            else:
                names.append(re.search(r"(\w*)\s*$", text[:i]).group(1))
    return names


@pytest.mark.parametrize("name", ["mla_decode.cu", "mla_prefill.cu"])
def test_a_warp_tests_a_barrier_by_a_vote(name):
    """In these kernels a whole warp issues the MMAs.  A barrier's phase may complete between two lanes'
    tests, so a branch on a test has to be on the warp's vote of it: lanes that branch apart would meet in
    different warp-wide operations, which is undefined and may never end."""
    text = _code(name)
    for m in re.finditer(r"\bmbar_test_wait\s*\(", text):
        assert "__all_sync" in _enclosing_calls(text, m.start()), text[max(0, m.start() - 80):m.end() + 60]


def test_the_check_sees_an_unvoted_test():
    assert _enclosing_calls("if (!f(a) && g(h(X", 17) == ["h", "g", "if"]
    assert "__all_sync" not in _enclosing_calls("x; if (!mbar_test_wait(b, p)) ok", 8)

"""Checks of the grouped-head kernels' sources for mistakes that a run shows only by chance (no GPU needed)."""
import re

import pytest

from test_kernel_sources import _code, _enclosing_calls


@pytest.mark.parametrize("name", ["gqa_decode.cu", "gqa_prefill.cu"])
def test_a_warp_tests_a_barrier_by_a_vote(name):
    """A whole warp issues the MMAs: a branch on a barrier's test has to be on the warp's vote of it."""
    text = _code(name)
    for m in re.finditer(r"\bmbar_test_wait\s*\(", text):
        assert "__all_sync" in _enclosing_calls(text, m.start()), text[max(0, m.start() - 80):m.end() + 60]


@pytest.mark.parametrize("name", ["gqa_decode.cu", "gqa_prefill.cu", "kv_write.cu", "pages.cu"])
def test_every_wait_is_bounded(name):
    """Waits on barriers in memory go through the bounded mbar_wait."""
    assert not re.search(r"mbarrier|try_wait|while\s*\(\s*!\s*mbar", _code(name))

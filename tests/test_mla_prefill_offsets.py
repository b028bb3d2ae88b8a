"""Query offsets of prompt attention that are not what the header asks for: what is reported, and which
requests are written all the same."""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_mla_prefill import _case, _run

pytestmark = pytest.mark.gpu

# Keys by the block, and (few heads, many keys) shared by the CTAs of clusters.
SHAPES = [([100, 300, 50], [100, 300, 50], 4), ([100, 300, 50], [4100, 4300, 4050], 8)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _with(c, offsets):
    return {**c, "cu_q": torch.tensor(offsets, dtype=torch.int32, device="cuda"), "max_q": 300}


@pytest.mark.parametrize("qlens,klens,H", SHAPES)
@pytest.mark.parametrize("offsets", [[0, 300, 250, 450], [0, 10 ** 6, 50, 200], [0, 100, 99, 450],
                                     [450, 100, 400, 450], [0, 400, 400, 0], [0, 100, -1, 450]])
def test_decreasing_offsets_skip_the_call(qlens, klens, H, offsets):
    """Requests of such offsets share rows: nothing is written, and the error is raised."""
    out, lse = _run(_with(_case(qlens, klens, H, seed=11), offsets), True)
    assert api.dsa_get_device_error() == 5
    assert (out == 77).all() and (lse == 77).all()


@pytest.mark.parametrize("qlens,klens,H", SHAPES)
def test_offsets_outside_skip_their_request(qlens, klens, H):
    c = _case(qlens, klens, H, seed=12)
    good, e_good = _run(c, True)
    assert api.dsa_get_device_error() == 0
    for offsets, kept in (([0, 100, 400, 10 ** 6], [(0, 400)]), ([0, 100, 10 ** 6, 2 ** 31 - 1], [(0, 100)]),
                          ([-1, 100, 400, 450], [(100, 450)]), ([-2 ** 31, -7, 400, 450], [(400, 450)])):
        out, lse = _run(_with(c, offsets), True)
        assert api.dsa_get_device_error() == 5
        left = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
        for a, b in kept:
            assert torch.equal(out[a:b], good[a:b]) and torch.equal(lse[a:b], e_good[a:b]), (offsets, a, b)
            left[a:b] = False
        assert (out[left] == 77).all() and (lse[left] == 77).all(), offsets


def test_a_request_outside_that_has_no_block_of_the_grid():
    """One query row in all: the grid has one block, the first request's."""
    c = _case([1], [9], 2, seed=13, tail=0)
    good, _ = _run(c, True)
    two = {**c, "cu_q": torch.tensor([0, 1, 500], dtype=torch.int32, device="cuda"),
           "cu_k": torch.tensor([0, 9, 9], dtype=torch.int32, device="cuda")}
    out, _ = _run(two, True)
    assert api.dsa_get_device_error() == 5 and torch.equal(out, good)


def test_many_requests_one_decreasing_offset():
    """The last of 3000 requests, and one of every place in the threads' walk."""
    n = 3000
    c = _case([2] * n, [2] * n, 1, seed=14, tail=0)
    good, _ = _run(c, True)
    assert api.dsa_get_device_error() == 0
    for r in (1, 64, 65, 511, 1024, n - 1, n):
        offsets = c["cu_q"].clone()
        offsets[r] = offsets[r - 1] - 1
        out, lse = _run({**c, "cu_q": offsets}, True)
        assert api.dsa_get_device_error() == 5, r
        assert (out == 77).all() and (lse == 77).all(), r
    again, _ = _run(c, True)
    assert api.dsa_get_device_error() == 0 and torch.equal(again, good)

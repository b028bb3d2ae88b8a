"""Attention over FP8 rows at the end of the range that value scales of a request may have: 2^100 from the least to the
largest.  Tolerances as in the test of the formula; the sum (the log-sum-exp, and the denominator of every output) has
the weights of rows of the least scale whole: P of them is 2^-100 of the largest or less, P / scale is not."""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_gqa_decode_fp8 import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("nq,H,K", [(1, 8, 1), (2, 16, 2), (1, 32, 1), (4, 32, 2), (1, 128, 1)])
@pytest.mark.parametrize("low,high,every", [(-80, 20, 50), (-80, 20, 2), (-80, 20, 1000), (-60, 40, 17), (-20, 80, 301)])
def test_scales_two_to_the_100_apart(nq, H, K, low, high, every):
    """One row in `every` has the largest scale, the others the least."""
    c = _case([2500, 300, 129], nq, H, K, seed=every + H, spread=2)
    for r, n in enumerate(c["lens"]):
        at = c["table"][r, :-(-n // 64)].long()
        s = torch.full((len(at) * 64, K), float("nan"), device="cuda")
        s[:n] = 2.0 ** low
        s[every // 2:n:every] = 2.0 ** high
        c["vs"][at] = s.unflatten(0, (len(at), 64)).transpose(1, 2)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=(0, H // 2, H - 1))

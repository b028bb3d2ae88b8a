"""Dense latent attention over FP8 rows against the formula over the rows as they are multiplied.

FP8 rows: a value is its code times its scale in fp32, rounded to bf16.  Rounding the float64 formula's keys
the same way leaves the kernel only the roundings that it makes for bf16 rows, so that their tolerance holds
(tests/test_mla_dense.py) without a term for the keys.  That term, 2^-8 of the sum of a score's 576 products'
sizes, would allow outputs of half their size over many keys.
"""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_mla_dense import CASES, JOINS, SM, _case, _check, _fp8, _run


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _rounded_rows(c):
    """(case, cache): the case over FP8 rows, its keys as the kernel multiplies them."""
    case, kv8 = _fp8(c)
    table = case["keep"][1].cpu()
    keys = []
    for r, n in enumerate(case["lens"]):
        pos = torch.arange(n)
        x = kv8[(table[r, pos // 64].long() * 64 + pos % 64).cuda()]
        sc = x[:, 512:528].contiguous().view(torch.float32).repeat_interleave(128, dim=1)
        value = (x[:, :512].contiguous().view(torch.float8_e4m3fn).float() * sc).to(torch.bfloat16)
        keys.append(torch.cat([value, x[:, 528:].contiguous().view(torch.bfloat16)], dim=1))
    return {**case, "keys": keys}, kv8


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nq,H", CASES + JOINS)
def test_fp8_rows_match_the_formula_of_rounded_rows(L, lens, nq, H):
    case, kv8 = _rounded_rows(_case(lens, nq, H, seed=len(lens) * 31 + nq * 7 + H))
    out, lse = _run(case, call=api.dsa_mla_decode_fp8kv, kv=kv8)
    assert api.dsa_get_device_error() == 0
    _check(case, out, lse)


@pytest.mark.parametrize("n,H", [(4097, 128), (9000, 64), (20000, 32), (40000, 16)])
def test_the_tolerance_shows_a_wrong_result(n, H):
    """(On the CPU.)  Outputs of the formula pass; three quarters of them, and those without the last
    fiftieth of the keys, do not."""
    g = torch.Generator().manual_seed(n)
    H = min(H, 4)
    q = torch.randn(1, H, 576, generator=g).to(torch.bfloat16)
    k = torch.randn(n, 576, generator=g).to(torch.bfloat16)
    c = dict(q=q, keys=[k], lens=[n], nq=1, H=H)

    def formula(keys):
        x = SM * (q[0].double() @ keys.double().T)
        lse = torch.logsumexp(x, 1)
        return (torch.exp(x - lse[:, None]) @ keys[:, :512].double())[None], lse[None]

    out, lse = formula(k)
    _check(c, out.to(torch.bfloat16), lse.float())
    with pytest.raises(AssertionError):
        _check(c, 0.75 * out, None)
    fewer, fewer_lse = formula(k[:n - n // 50])
    with pytest.raises(AssertionError):
        _check(c, fewer, None)
    with pytest.raises(AssertionError):
        _check(c, out, fewer_lse)

"""Dense latent attention where scores span many powers of two, and FP8 rows against the formula over the
rows as they are multiplied.

FP8 rows: a value is its code times its scale in fp32, rounded to bf16.  Rounding the float64 formula's keys
the same way leaves the kernel only the roundings that it makes for bf16 rows, so that their tolerance holds
(tests/test_mla_dense.py) without a term for the keys.  That term, 2^-8 of the sum of a score's 576 products'
sizes, would allow outputs of half their size over many keys.
"""
import math

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


# Scores (natural logarithms) that a position adds through the last rope dim: rising by ten powers of two a
# 128-token tile, falling as fast, and rising in waves.
RAMPS = {
    "rise": lambda t: t * (10 * math.log(2) / 128),
    "fall": lambda t: -t * (10 * math.log(2) / 128),
    "waves": lambda t: t * (3 * math.log(2) / 128) + 25 * torch.sin(t / 90),
}
STEP = 16.0     # the queries' value in that dim


def _ramped(lens, nq, H, ramp, seed):
    c = _case(lens, nq, H, seed)
    c["q"][..., 575] = STEP
    table = c["keep"][1].cpu()
    for r, n in enumerate(lens):
        t = torch.arange(n)
        c["keys"][r][:, 575] = (RAMPS[ramp](t.float()) / (STEP * SM)).to(torch.bfloat16).cuda()
        c["kv"][(table[r, t // 64].long() * 64 + t % 64).cuda()] = c["keys"][r]
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("lens,nq,H", [
    ([3000] * 40, 1, 128),            # stretches of 13 tiles of bf16 rows, 25 of FP8 rows
    ([2900, 3100] * 20, 2, 128),      # of 26, 50
    ([20000] * 2, 1, 16),             # of 4, 8: parts whose weights differ by up to 2^1500
    ([6000, 300, 9000], 3, 96),
])
def test_scores_over_many_powers_of_two(L, lens, nq, H, ramp, fp8):
    c = _ramped(lens, nq, H, ramp, seed=len(lens) + nq + H)
    if ramp != "fall":
        # The running maximum over a request's tiles rises by more than 2^8 again and again.
        x = SM / math.log(2) * (c["q"][0].double() @ c["keys"][0].double().T)
        tops = torch.stack([p.amax(1) for p in x.split(128, dim=1)], dim=1)
        run = torch.cummax(tops, dim=1).values
        assert ((run[:, 1:] - run[:, :-1]) > 8).sum(1).min() >= (8 if ramp == "rise" else 2)
    call, cache = api.dsa_mla_decode, None
    if fp8:
        c, cache = _rounded_rows(c)
        call = api.dsa_mla_decode_fp8kv
    out, lse = _run(c, call=call, kv=cache)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse)
    again, _ = _run(c, lse=False, call=call, kv=cache)
    assert torch.equal(out, again)

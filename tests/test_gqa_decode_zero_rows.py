"""Attention over FP8 rows where some value rows are zeros (a sink's, padding's), which dsa_kv_write_fp8 gives scale 1,
among rows of small values, whose scales are far below it.

Tolerances, derived beforehand, as in the test of the formula (its A, dx and z) but for what a cut of the weights may
take: a weight times its scale is held to 2^-29 of the largest weight times scale of the request (more than 16 rows:
2^-32, half a step of 2^-31), where rows of zeros count with 2^-80.  With c_s the scales and p_s the weights, out is off
by 2^-8 |out| + (2^-11 + 2.1 dx + n 2^-24 + 2^-18) A + 2^-29 max_s(p_s c_s) sum_s |code_s|: nothing in it depends on the
scale that rows of zeros have in the cache.  z of a row of zeros is |x| / ln 2 + 80.
"""
import math

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_gqa_decode_fp8 import D, _case, _run

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _written(lens, nq, H, K, size, lead, zeros, seed, minus=False):
    """Requests as the cache write makes them: keys of scores N(0, 1), values |N(0, size^2)|; the rows `zeros(r)` have
    zero values, and keys that every query scores with `lead`."""
    c = _case(lens, nq, H, K, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    c["q"].copy_(torch.randn(c["q"].shape, generator=g, device="cuda"))
    c["q"][..., 0] = 8.0
    for r, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (torch.randn(n, K, D, generator=g, device="cuda") for _ in range(2))
        v = v.abs() * size
        z = torch.zeros(n, dtype=torch.bool, device="cuda")
        z[zeros(r)] = True
        k[..., 0] = 0.0
        k[z] = 0.0
        k[z, :, 0] = lead * D ** 0.5 / 8.0
        v[z] = -0.0 if minus else 0.0
        i = torch.arange(n, device="cuda")
        slots = (c["table"][r].long()[i // 64] * 64 + i % 64).to(torch.int32)
        api.dsa_kv_write_fp8(k.to(torch.bfloat16), v.to(torch.bfloat16), slots, c["k"], c["ks"], c["v"], c["vs"])
    return c


def _check(c, out, lse, heads):
    nq, G = c["nq"], c["H"] // c["K"]
    sm = D ** -0.5
    for r, n in enumerate(c["lens"]):
        at = c["table"][r, :-(-n // 64)].long()
        for h in heads:
            code, scale = ([c[x][at, h // G].flatten(0, 1)[:n].view(torch.float8_e4m3fn).double() for x in "kv"],
                           [c[x][at, h // G].flatten()[:n].double() for x in ("ks", "vs")])
            k, v = code[0] * scale[0][:, None], code[1] * scale[1][:, None]
            zero = (code[1] == 0).all(dim=1)
            assert (scale[1][zero] == 1).all()
            cs = torch.where(zero, 2.0 ** -80, scale[1])
            q = c["q"][r * nq:(r + 1) * nq, h].double()
            lim = n - nq + 1 + torch.arange(nq, device="cuda")
            hide = torch.arange(n, device="cuda")[None, :] >= lim[:, None]
            x = (sm * (q @ k.T)).masked_fill(hide, -INF)
            E = (sm * (q.abs() @ k.abs().T)).masked_fill(hide, 0.0).amax(1)
            Q = (sm * q.abs().amax(1)[:, None] * k.abs().sum(1)[None, :]).masked_fill(hide, 0.0).amax(1)
            z = (x.abs() / math.log(2) + torch.log2(cs).abs()[None, :]).masked_fill(hide, 0.0).amax(1)
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            dx = 258 * 2.0 ** -24 * E + 2.0 ** -17 * Q + 2.0 ** -21 * z
            ref, A = p @ v, p @ v.abs()
            cut = 2.0 ** -29 * (p * cs[None, :]).amax(1)[:, None] * code[1].abs().sum(0)[None, :]
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.1 * dx[:, None] + n * 2.0 ** -24 + 2.0 ** -18) * A + cut
            got, e_got = out[r * nq:(r + 1) * nq, h].double(), lse[r * nq:(r + 1) * nq, h].double()
            assert ((got - ref).abs() <= tol).all(), (r, n, h, ((got - ref).abs() / tol).nan_to_num(0).max(),
                                                      (got - ref).norm() / ref.norm())
            assert ((e_got - e).abs() <= dx + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * e.abs()).all(), (r, n, h)


# 8, 16, 32, 64 and 128 rows of a key head: each way that the kernel reads them.
ROWS = [(1, 8, 1), (2, 16, 2), (1, 32, 1), (4, 32, 2), (1, 128, 1)]
PLACES = {"first": lambda r: slice(0, 1), "inside": lambda r: [130 + r], "a tile": lambda r: slice(0, 128),
          "end": lambda r: slice(-4, -3), "every fifth": lambda r: slice(3, None, 5)}


@pytest.mark.parametrize("nq,H,K", ROWS)
@pytest.mark.parametrize("size,lead", [(0.02, 8.0), (0.02, 10.0), (1e-3, 8.0), (1e-6, 14.0)])
def test_one_row_of_zeros(nq, H, K, size, lead):
    c = _written([4096, 301], nq, H, K, size, lead, PLACES["first"], seed=H + nq)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=(0, H // 2, H - 1))


@pytest.mark.parametrize("nq,H,K", ROWS)
@pytest.mark.parametrize("place", PLACES)
def test_where_the_zeros_lie(nq, H, K, place):
    c = _written([5000, 700, 64 * 9], nq, H, K, 1e-3, 9.0, PLACES[place], seed=3 * H + nq, minus=place == "inside")
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=(0, H - 1))


@pytest.mark.parametrize("nq,H,K", ROWS)
def test_nothing_but_zeros(nq, H, K):
    """Outputs of zeros; the sum holds every weight."""
    c = _written([1000, 130], nq, H, K, 1.0, 3.0, lambda r: slice(None), seed=H)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    assert (out == 0).all()
    _check(c, out, lse, heads=(0, H - 1))


@pytest.mark.parametrize("nq,H,K", ROWS)
def test_scale_one_without_zeros(nq, H, K):
    """Rows whose largest value is 448 have scale 1 too, and count as any other."""
    c = _written([900, 200], nq, H, K, 1.0, 0.0, lambda r: slice(0, 0), seed=H + 5)
    for r, n in enumerate(c["lens"]):
        i = torch.arange(2, n, 7, device="cuda")
        v = torch.zeros(len(i), K, D, device="cuda", dtype=torch.bfloat16)
        v[torch.arange(len(i)), :, torch.arange(len(i)) % D] = 448.0          # one value of the row
        slots = (c["table"][r].long()[i // 64] * 64 + i % 64).to(torch.int32)
        k = torch.randn(len(i), K, D, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
        k[..., 0] = 0.0
        api.dsa_kv_write_fp8(k.to(torch.bfloat16), v, slots, c["k"], c["ks"], c["v"], c["vs"])
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=(0, H - 1))


def test_the_same_outputs_whatever_scale_the_zeros_were_given():
    """Scale 1, as the cache write gives it, and the least that scales count as: the same bits."""
    c = _written([3000], 1, 8, 1, 1e-3, 9.0, PLACES["every fifth"], seed=2)
    out, lse = _run(c)
    c["vs"][c["vs"] == 1.0] = 2.0 ** -80
    small, lse_small = _run(c)
    assert api.dsa_get_device_error() == 0
    assert torch.equal(out, small) and torch.equal(lse, lse_small)

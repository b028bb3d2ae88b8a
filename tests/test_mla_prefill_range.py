"""Prompt attention where scores span many powers of two: the running maximum rises again and again, and the
parts of an item whose keys the CTAs of a cluster share have weights far apart."""
import math

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_mla_prefill import SHARED, SM, _case, _check, _run

pytestmark = pytest.mark.gpu

# Scores (natural logarithms) that a key's position in its request adds through the last rope dim: rising by ten
# powers of two a 128-key tile, falling as fast, and rising in waves.
RAMPS = {
    "rise": lambda t: t * (10 * math.log(2) / 128),
    "fall": lambda t: -t * (10 * math.log(2) / 128),
    "waves": lambda t: t * (3 * math.log(2) / 128) + 25 * torch.sin(t / 90),
}
STEP = 16.0     # the queries' value in that dim


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("qlens,klens,H", SHARED + [([1500, 700], [1500, 2500], 6), ([900] * 8, [900] * 8, 40)])
def test_scores_over_many_powers_of_two(qlens, klens, H, ramp, causal):
    build.build()
    c = _case(qlens, klens, H, seed=sum(qlens) * 3 + sum(klens) + H)
    c["q"][:sum(qlens), :, 191] = STEP
    at = 0
    for m in klens:
        t = torch.arange(m, dtype=torch.float32, device="cuda")
        c["rope"][at:at + m, 63] = (RAMPS[ramp](t) / (STEP * SM)).to(torch.bfloat16)
        at += m
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse, heads=range(0, H, max(1, H // 4)))
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)

"""The residual + root-mean-square norm at the ends of fp32's range: tiles whose y is zero although their
values are not."""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

pytestmark = pytest.mark.gpu


def _codes(x, w, eps, group):
    build.build()
    rows, dim = x.shape
    y, y8 = torch.empty_like(x), torch.empty((rows, dim), dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, -(-dim // 128) if group else 1), 33.0, device="cuda")
    api.dsa_rmsnorm(x, w, eps, y=y, y8=y8, y_scale=sc, group=group)
    alone, sc_alone = torch.empty_like(y8), torch.empty_like(sc)
    api.dsa_rmsnorm(x, w, eps, y8=alone, y_scale=sc_alone, group=group)
    assert torch.equal(y8, alone) and torch.equal(sc, sc_alone)
    return y.float(), y8.view(torch.float8_e4m3fn).float(), sc


@pytest.mark.parametrize("dim", [256, 1032, 4104])
@pytest.mark.parametrize("group", [0, 128])
def test_a_sum_of_squares_past_the_range(dim, group):
    """y = h / inf = 0: scale 1 and codes 0, for the tiles of such a row and no others."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(4, dim, generator=g, device="cuda")
    x[1] *= 1e20
    x[3, dim - 1] = 3e38                      # one value is enough
    x = x.to(torch.bfloat16)
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    y, codes, sc = _codes(x, w, 1e-6, group)
    assert (y[[1, 3]] == 0).all() and (codes[[1, 3]] == 0).all() and (sc[[1, 3]] == 1).all()
    assert (y[[0, 2]] != 0).any(1).all() and (sc[[0, 2]] < 1).all() and codes[[0, 2]].abs().amax() == 448


@pytest.mark.parametrize("group", [0, 128])
def test_values_that_round_to_zero(group):
    """h * weight = 2^-149, the smallest fp32 value, and rms = 1000: y = 0."""
    x = torch.full((2, 256), 2.0 ** -130, dtype=torch.bfloat16, device="cuda")
    w = torch.full((256,), 2.0 ** -19, dtype=torch.bfloat16, device="cuda")
    y, codes, sc = _codes(x, w, 1e6, group)
    assert (y == 0).all() and (codes == 0).all() and (sc == 1).all()

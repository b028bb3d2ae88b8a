"""Prompt attention: refusals of sizes, on the host."""
import pytest

from deepseek_sparse_attention_lightning_gb300 import api, build

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


@pytest.mark.parametrize("batch,heads,total_q", [
    (1, 1024, 2 ** 31 - 1), (65535, 1024, 536800000), (1, 256, 2 ** 31 - 1),
])
def test_a_grid_past_31_bits_is_unsupported(L, batch, heads, total_q):
    assert (total_q + 255 * batch) // 256 * heads > 2 ** 31 - 1
    assert L.dsa_mla_prefill(batch, heads, total_q, 64, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 576, 0.07, 1, FAKE, None,
                             None) == 2

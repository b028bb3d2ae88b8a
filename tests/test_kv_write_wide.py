"""The cache write of tokens that are wider than a block of threads (more than 16 heads of 128 bf16 dims, 32 of FP8 or
of 64 dims): several passes over a token, the last of them with part of a warp.  Bits as in the tests of the write."""
import pytest
import torch

import test_kv_write as narrow
from deepseek_sparse_attention_lightning_gb300 import api, build

pytestmark = pytest.mark.gpu
SIZES = [(65, 33, 128, 2, 8), (9, 100, 128, 1, 0), (130, 17, 128, 3, 0), (40, 65, 128, 1, 24), (70, 33, 64, 2, 8), (3, 1024, 64, 1, 0),
         (3, 1024, 128, 1, 0), (5, 1023, 128, 1, 8), (1, 20, 128, 1, 0), (33, 31, 128, 1, 8)]


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


@pytest.mark.parametrize("T,K,D,pages,wide", SIZES)
def test_bf16_rows_are_copied(L, T, K, D, pages, wide):
    narrow.test_bf16_rows_are_copied(L, T, K, D, pages, wide)


@pytest.mark.parametrize("T,K,D,pages,wide", [s for s in SIZES if s[2] == 128])
def test_fp8_rows(L, T, K, D, pages, wide):
    narrow.test_fp8_rows(L, T, K, D, pages, wide)


@pytest.mark.parametrize("T,K,pages", [(65, 33, 2), (5, 1023, 1), (1000, 8, 16), (77, 3, 2)])
def test_codes_are_those_of_the_division(L, T, K, pages):
    """amax / 448 and x / scale in fp32, rounded to E4M3: the same bits, skipped tokens left as they were."""
    k, v, slots = narrow._case(T, K, 128, pages, 0, T + K)
    slots[T // 3] = -1
    live = slots >= 0
    codes = [torch.full((pages, K, 64, 128), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, K, 64), 77.0, device="cuda") for _ in range(2)]
    api.dsa_kv_write_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    assert api.dsa_get_device_error() == 0
    for x, c, s in zip((k, v), codes, scales):
        x = x[live].float()
        top = x.abs().amax(dim=2)
        scale = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))
        want = torch.full((pages * 64, K, 128), 77, dtype=torch.uint8, device="cuda")
        want[slots[live].long()] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        want_s = torch.full((pages * 64, K), 77.0, device="cuda")
        want_s[slots[live].long()] = scale
        assert torch.equal(c.transpose(1, 2).flatten(0, 1), want)
        assert torch.equal(s.transpose(1, 2).flatten(0, 1), want_s)

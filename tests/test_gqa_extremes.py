"""The grouped-head attentions at the ends of what they take: many heads, many requests, one very long request, queries
of zeros, and a workspace that is exactly large enough.  Tolerances as in the tests of each."""
import pytest
import torch

import test_gqa_decode as dec
import test_gqa_decode_fp8 as dec8
import test_gqa_prefill as pre
from deepseek_sparse_attention_lightning_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("H,K,D", [(1024, 8, 64), (1024, 1024, 64), (512, 8, 128), (1000, 125, 128)])
def test_many_heads(H, K, D):
    c = pre._case([3, 40], [5, 200], H, K, D, seed=H + K)
    out, lse = pre._run(c, True)
    assert api.dsa_get_device_error() == 0
    pre._check(c, True, out, lse, heads=range(0, H, H // 7))


def test_as_many_requests_as_there_may_be():
    """65535 prompts of one or two queries over a few keys: each against the mean of its equal-scored values."""
    B, H, K, D = 65535, 16, 2, 64
    n = 1 + torch.arange(B) % 2
    m = n + torch.arange(B) % 5
    cu = lambda x: torch.cat([torch.zeros(1, dtype=torch.int64), x.cumsum(0)]).to(torch.int32).cuda()
    Tq, Tk = int(n.sum()), int(m.sum())
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.zeros((Tq, H, D), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn(Tk, K, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((Tq, H), device="cuda")
    api.dsa_gqa_prefill(q, k, v, cu(n), cu(m), out, 2, 0.1, lse=lse)
    assert api.dsa_get_device_error() == 0
    # Scores are 0: the last query sees all m keys, the one before m - 1.
    sums = torch.cat([torch.zeros(1, K, D, dtype=torch.float64, device="cuda"), v.double().cumsum(0)])
    sizes = torch.cat([torch.zeros(1, K, D, dtype=torch.float64, device="cuda"), v.double().abs().cumsum(0)])
    rq = torch.repeat_interleave(torch.arange(B), n)
    i = torch.arange(Tq) - cu(n).cpu().long()[rq]
    seen = (m[rq] - n[rq] + i + 1).cuda()
    lo = cu(m).long()[rq.cuda()]
    mean = lambda s: (s[lo + seen] - s[lo]) / seen[:, None, None]
    want, A = mean(sums).repeat_interleave(H // K, 1), mean(sizes).repeat_interleave(H // K, 1)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -18) * A + 1e-9).all()
    assert ((lse.double() - seen.double().log()[:, None]).abs() <= 2.0 ** -19).all()


@pytest.mark.parametrize("D", [64, 128])
def test_one_very_long_request(D):
    c = dec._case([1500001], 2, 8, 1, D, seed=D, extra_pages=1)
    out, lse = dec._run(c)
    assert api.dsa_get_device_error() == 0
    dec._check(c, out, lse, heads=[0, 7])


def test_one_very_long_request_fp8():
    c = dec8._case([1500001], 1, 5, 1, seed=3, extra_pages=1)
    out, lse = dec8._run(c)
    assert api.dsa_get_device_error() == 0
    dec8._check(c, out, lse)


@pytest.mark.parametrize("nq,H,K", [(1, 8, 2), (3, 60, 2), (1, 128, 1)])
def test_queries_of_zeros(nq, H, K):
    c = dec8._case([500, 70], nq, H, K, seed=4)
    c["q"].zero_()
    out, lse = dec8._run(c)
    assert api.dsa_get_device_error() == 0
    dec8._check(c, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_an_exact_workspace_is_not_overrun(fp8):
    mod = dec8 if fp8 else dec
    args = ([3000, 900], 4, 128, 1)
    c = mod._case(*args, seed=5) if fp8 else mod._case(*args, 128, seed=5)
    n = c["ws"].numel()
    buf = torch.full((n + 4096,), 170, dtype=torch.uint8, device="cuda")
    want, _ = mod._run(c)
    got, _ = mod._run({**c, "ws": buf[:n]})
    assert api.dsa_get_device_error() == 0
    assert torch.equal(got, want) and (buf[n:] == 170).all()


def test_prompts_of_one_query_agree_with_decode():
    """One query over packed keys, and the same over the cache: two kernels, one formula."""
    c = dec._case([700, 64, 1, 2000], 1, 40, 8, 128, seed=6)
    got, e = dec._run(c)
    k, v = (torch.cat([torch.cat([dec.rows_of(c, c[x], r, h, n)[:, None] for h in range(8)], 1) for r, n in enumerate(c["lens"])])
            for x in "kv")
    cu = lambda n: torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(got), torch.empty_like(e)
    api.dsa_gqa_prefill(c["q"], k, v, cu([1] * 4), cu(c["lens"]), out, 1, 128 ** -0.5, lse=lse)
    assert api.dsa_get_device_error() == 0
    assert (lse - e).abs().max() <= 1e-4
    assert ((out.float() - got.float()).abs() <= 2.0 ** -6 * got.float().abs() + 2.0 ** -7).all()

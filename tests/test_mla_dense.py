"""Dense latent attention over the paged cache (absorbed form), against its formula in float64.

Tolerances, fixed beforehand.  With A = sum_s p_s |v_s| (the exact probabilities) and E the largest
sm_scale * sum_d |q_d c_d| of a row's visible keys:
  * scores: 576 products accumulated in fp32, at most 576 roundings of 2^-24 of E each: dx = 576 * 2^-24 * E;
  * probabilities are rounded to bf16 (half a step, 2^-8) and carry exp(dx) - 1 from the scores, in
    numerator and sum: (2^-8 + 2.1 dx) * A; the fp32 accumulation over n keys n * 2^-24 * A; the
    joining of partials and the normalisation 2^-18 * A;
  * the output is rounded to bf16: 2^-8 |out|.
  * log-sum-exp: dx + n * 2^-24 (sum of n terms) + 2^-20 (exponential and logarithm) + 2^-23 |lse|.
FP8 rows: codes are multiplied by their scale and rounded to bf16, so a key or value is off by
2^-8 of itself: dx grows by 2^-8 E, the output by 2^-8 A.
"""
import ctypes

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

SM = 1.0 / 192.0 ** 0.5
FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _fake_desc(**over):
    d = dict(batch=2, q_per_req=1, num_heads=128, topk=0, page_size=64, max_pages=4, num_pages=8,
             seqlens=0x10000, page_table=0x20000)
    d.update(over)
    return api.DecodeDesc(**d)


def test_refusals_on_the_host(L):
    need = L.dsa_mla_decode_workspace_bytes(ctypes.byref(_fake_desc()))
    assert need > 0

    def call(desc=None, q=FAKE, kv=FAKE, scale=SM, out=FAKE, lse=FAKE, ws=FAKE, nbytes=need, **over):
        d = ctypes.byref(_fake_desc(**over)) if desc is None else desc
        return L.dsa_mla_decode(d, q, kv, scale, out, lse, ws, nbytes, None)

    assert L.dsa_mla_decode(None, FAKE, FAKE, SM, FAKE, None, FAKE, need, None) == 1
    for bad in (dict(q=None), dict(kv=None), dict(out=None), dict(q=FAKE + 8), dict(kv=FAKE + 8),
                dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(batch=0), dict(num_heads=0),
                dict(q_per_req=0), dict(seqlens=None), dict(page_table=0x20002), dict(num_pages=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(num_heads=129), dict(q_per_req=5), dict(batch=1025), dict(page_size=32),
                dict(num_pages=1 << 25)):
        assert call(**bad) == 2, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(nbytes=need - 1)):
        assert call(**bad) == 3, bad
    assert L.dsa_mla_decode_workspace_bytes(ctypes.byref(_fake_desc(num_heads=129))) == 0
    assert L.dsa_mla_decode_workspace_bytes(None) == 0


def _case(lens, nq, H, seed, spare=3, scale=1.0):
    """A paged cache whose unused rows (other pages, rows behind a request's end) hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [(n + 63) // 64 for n in lens]
    num_pages = sum(pages) + spare
    max_pages = max(1, max(pages)) + 1
    phys = torch.randperm(num_pages, generator=host).to(torch.int32)
    table = torch.full((B, max_pages), 0x7fffffff, dtype=torch.int32)      # never read past the end
    kv = torch.full((num_pages * 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    keys, at = [], 0
    for r, n in enumerate(lens):
        table[r, :pages[r]] = phys[at:at + pages[r]]
        at += pages[r]
        pos = torch.arange(n)
        rows = (table[r, pos // 64].long() * 64 + pos % 64).cuda()
        c = (torch.randn(n, 576, generator=g, device="cuda") * scale).to(torch.bfloat16)
        kv[rows] = c
        keys.append(c)
    q = torch.randn(B * nq, H, 576, generator=g, device="cuda").to(torch.bfloat16)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = table.cuda()
    desc = api.make_desc(seq, table, nq, H, 1, num_pages)
    return dict(desc=desc, q=q, kv=kv, keys=keys, lens=lens, nq=nq, H=H, keep=(seq, table))


def _run(c, lse=True, stream=None, call=None, kv=None):
    T, H = c["q"].shape[:2]
    out = torch.full((T, H, 512), 77.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full((T, H), 77.0, device="cuda") if lse else None
    ws = torch.empty(api.dsa_mla_decode_workspace_bytes(c["desc"]), dtype=torch.uint8, device="cuda")
    (call or api.dsa_mla_decode)(c["desc"], c["q"], c["kv"] if kv is None else kv, out, ws, SM, lse=e,
                                 stream=stream)
    return out, e


def _check(c, out, lse, rel_key=0.0):
    nq, H = c["nq"], c["H"]
    for r, n in enumerate(c["lens"]):
        k = c["keys"][r].double()
        for i in range(nq):
            t = r * nq + i
            vis = max(0, n - (nq - 1 - i))
            got = out[t].double()
            if vis == 0:
                assert (got == 0).all()
                assert lse is None or (lse[t] == float("-inf")).all()
                continue
            q, kk = c["q"][t].double(), k[:vis]
            x = SM * (q @ kk.T)
            E = (SM * (q.abs() @ kk.abs().T)).amax(1)
            dx = (576 * 2.0 ** -24 + rel_key) * E
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            ref, A = p @ kk[:, :512], p @ kk[:, :512].abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel_key + 2.1 * dx[:, None] + vis * 2.0 ** -24 + 2.0 ** -18) * A
            assert ((got - ref).abs() <= tol).all(), (r, i, ((got - ref).abs() / tol).max())
            if lse is not None:
                bound = dx + vis * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * e.abs()
                assert ((lse[t].double() - e).abs() <= bound).all(), (r, i)


CASES = [
    ([1], 1, 128), ([1], 1, 1), ([2, 1], 2, 16), ([0], 1, 16), ([0, 5, 0, 64, 0], 1, 48),
    ([63, 64, 65, 128, 127, 1], 1, 128), ([31, 32, 33], 3, 16), ([3, 1, 0, 2], 4, 128),
    ([4096], 1, 16), ([4097], 1, 128), ([777, 2049], 2, 128), ([1500, 20, 3000], 3, 96),
    ([5000], 4, 80), ([1000, 999, 64], 4, 32), ([100] * 90, 1, 7), (list(range(0, 300, 7)), 2, 20),
    ([9000, 1, 9000], 1, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nq,H", CASES)
def test_matches_formula(L, lens, nq, H):
    c = _case(lens, nq, H, seed=len(lens) * 100 + nq * 10 + H)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse)
    again, _ = _run(c, lse=False)
    assert torch.equal(out, again)


def _fp8(c):
    """The case with its cache in FP8 rows; unused rows stay NaN codes with NaN scales."""
    kv8 = torch.full((c["kv"].shape[0], 656), 0xFF, dtype=torch.uint8, device="cuda")
    used = ~torch.isnan(c["kv"][:, 0])
    rows = torch.empty((int(used.sum()), 656), dtype=torch.uint8, device="cuda")
    api.dsa_latent_to_fp8(c["kv"][used].contiguous(), rows)
    kv8[used] = rows
    table, seq = c["keep"][1].cpu(), c["lens"]
    keys = []
    for r, n in enumerate(seq):
        pos = torch.arange(n)
        x = kv8[(table[r, pos // 64].long() * 64 + pos % 64).cuda()]
        sc = x[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, dim=1)
        codes = x[:, :512].contiguous().view(torch.float8_e4m3fn).double()
        keys.append(torch.cat([codes * sc, x[:, 528:].contiguous().view(torch.bfloat16).double()], dim=1))
    return {**c, "keys": keys}, kv8


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nq,H", CASES)
def test_fp8_rows_match_formula(L, lens, nq, H):
    c, kv8 = _fp8(_case(lens, nq, H, seed=len(lens) * 100 + nq * 10 + H))
    out, lse = _run(c, call=api.dsa_mla_decode_fp8kv, kv=kv8)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, rel_key=2.0 ** -8)
    again, _ = _run(c, lse=False, call=api.dsa_mla_decode_fp8kv, kv=kv8)
    assert torch.equal(out, again)


@pytest.mark.gpu
def test_large_scores_raise_the_maximum(L):
    """Keys that grow along the request: the running maximum rises by far more than 2^8 several times."""
    c = _case([1500], 1, 128, seed=3)
    ramp = (1.0 + torch.arange(1500, device="cuda") / 100.0)[:, None]
    c["keys"][0].copy_((c["keys"][0].float() * ramp).to(torch.bfloat16))
    table = c["keep"][1].cpu()
    pos = torch.arange(1500)
    c["kv"][(table[0, pos // 64].long() * 64 + pos % 64).cuda()] = c["keys"][0]
    out, lse = _run(c)
    _check(c, out, lse)

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


# Joins of many parts of few rows (FP8: twice the key tiles), of eight parts at a time, and of the
# few parts that many requests have.
JOINS = [
    ([40000], 1, 16), ([39999], 4, 16), ([20000, 30001], 1, 32), ([25000], 2, 128), ([700, 1300, 64] * 14, 1, 128),
    ([513] * 40, 2, 16), ([2000, 1] * 20, 1, 1), ([300, 1100] * 20, 3, 96),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,nq,H", JOINS)
def test_joins(L, lens, nq, H, fp8):
    c = _case(lens, nq, H, seed=len(lens) + nq + H)
    case, call, cache, rel = _both_caches(c)[fp8]
    out, lse = _run(case, call=call, kv=cache)
    assert api.dsa_get_device_error() == 0
    _check(case, out, lse, rel_key=rel)
    again, _ = _run(case, lse=False, call=call, kv=cache)
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


def _both_caches(c):
    fc, kv8 = _fp8(c)
    return ((c, api.dsa_mla_decode, c["kv"], 0.0), (fc, api.dsa_mla_decode_fp8kv, kv8, 2.0 ** -8))


@pytest.mark.gpu
def test_bad_page_ids_and_lengths_are_reported(L):
    """A page id outside the cache masks exactly its page's tokens; a length above the page table is cut
    to it; each is reported, and the rows of other requests stay right (bit for bit where the lengths, and
    with them the cuts between CTA pairs, are the same)."""
    c = _case([300, 200, 500], 1, 32, seed=9)
    seq, table = c["keep"]
    for case, call, cache, rel in _both_caches(c):
        good, _ = _run(case, call=call, kv=cache)
        assert api.dsa_get_device_error() == 0
        saved = table.clone()
        table[0, 1], table[2, 4] = -1, case["desc"].num_pages
        out, lse = _run(case, call=call, kv=cache)
        assert api.dsa_get_device_error() == 5
        assert torch.equal(out[1], good[1])
        keep0 = torch.cat([case["keys"][0][:64], case["keys"][0][128:]])
        keep2 = torch.cat([case["keys"][2][:256], case["keys"][2][320:]])
        _check({**case, "q": case["q"][[0, 2]], "keys": [keep0, keep2], "lens": [236, 436]}, out[[0, 2]], lse[[0, 2]], rel)
        table.copy_(saved)
        # the page table covers 9 pages (max_pages of this batch): 576 tokens
        seq[2] = 10 ** 6
        two = {**case, "q": case["q"][:2], "keys": case["keys"][:2], "lens": [300, 200]}
        out, lse = _run(case, call=call, kv=cache)
        assert api.dsa_get_device_error() == 5
        _check(two, out[:2], lse[:2], rel)
        seq[2] = -3
        out, lse = _run(case, call=call, kv=cache)
        assert api.dsa_get_device_error() == 0
        assert (out[2] == 0).all() and (lse[2] == float("-inf")).all()
        _check(two, out[:2], lse[:2], rel)
        seq[2] = 500
        again, _ = _run(case, call=call, kv=cache)
        assert api.dsa_get_device_error() == 0 and torch.equal(again, good)


@pytest.mark.gpu
def test_streams_and_graphs(L):
    """Two calls at once on two streams with workspaces of their own; a captured call replayed over new
    lengths, pages and queries."""
    c1, c2 = _case([4000, 100, 2500], 2, 64, seed=1), _case([70, 3000], 1, 128, seed=2)
    for (a, call, ca, _), (b, _, cb, _) in zip(_both_caches(c1), _both_caches(c2)):
        want_a, want_b = _run(a, call=call, kv=ca)[0], _run(b, call=call, kv=cb)[0]
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            for s, case, cache in ((s1, a, ca), (s2, b, cb)):
                with torch.cuda.stream(s):
                    got.append(_run(case, call=call, kv=cache, stream=s)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, want_a) for g in got[0::2]) and all(torch.equal(g, want_b) for g in got[1::2])

        seq, table = a["keep"]
        q0, seq0 = a["q"].clone(), seq.clone()
        a["q"].zero_()
        seq.fill_(2)
        out = torch.empty((6, 64, 512), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(api.dsa_mla_decode_workspace_bytes(a["desc"]), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(a["desc"], a["q"], ca, out, ws, SM)
        a["q"].copy_(q0)
        seq.copy_(seq0)
        graph.replay()
        assert torch.equal(out, want_a)
    assert api.dsa_get_device_error() == 0


@pytest.mark.gpu
def test_equals_the_sparse_layer_that_selects_everything(L):
    """With k >= the visible tokens the sparse decode layer attends them all: the same outputs, up to the
    rounding of both (each within its tolerance of the formula)."""
    from deepseek_sparse_attention_lightning_gb300 import workloads as W
    spec = W.small_spec("mtp_32k", batch=3, q_per_req=2, num_heads=128, topk=2048, heavy="none", seed=7)
    wl = W.make_workload(spec, seqlens=[1900, 64, 700]).to("cuda")
    sparse = api.run_decode(wl)
    T, H = spec.num_tokens, spec.num_heads
    desc = api.workload_desc(wl)
    out = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(api.dsa_mla_decode_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    api.dsa_mla_decode(desc, wl.q, wl.kv, out, ws, spec.sm_scale)
    assert api.dsa_get_device_error() == 0
    assert ((out.float() - sparse).abs() <= 2e-2 + 2e-2 * sparse.abs()).all()


@pytest.mark.gpu
def test_a_cache_past_two_to_the_31(L):
    """Rows whose byte and element offsets pass 32 bits, and a batch of 1024 requests."""
    g = torch.Generator(device="cuda").manual_seed(4)
    num_pages = 1 << 16                                  # 4.2 M rows, 2.4 G values
    for fp8 in (False, True):
        kv = torch.zeros((num_pages * 64, 656 if fp8 else 576), dtype=torch.uint8 if fp8 else torch.bfloat16,
                         device="cuda")
        lens = [1 + (37 * i) % 130 for i in range(1024)]
        table = torch.full((1024, 3), -1, dtype=torch.int32)
        page, keys = num_pages - 1, []
        for r, n in enumerate(lens):
            c = torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16)
            if fp8:
                rows = torch.empty((n, 656), dtype=torch.uint8, device="cuda")
                api.dsa_latent_to_fp8(c, rows)
                sc = rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, dim=1)
                keys.append(torch.cat([rows[:, :512].contiguous().view(torch.float8_e4m3fn).double() * sc,
                                       c[:, 512:].double()], dim=1))
            else:
                rows = c
                keys.append(c)
            for j in range(-(-n // 64)):
                table[r, j] = page
                part = rows[64 * j:64 * j + 64]
                kv[page * 64:page * 64 + part.shape[0]] = part
                page -= 1
        seq, table = torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()
        q = torch.randn(1024, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
        case = dict(desc=api.make_desc(seq, table, 1, 16, 1, num_pages), q=q, kv=kv, keys=keys, lens=lens, nq=1,
                    H=16, keep=(seq, table))
        out, lse = _run(case, call=api.dsa_mla_decode_fp8kv if fp8 else api.dsa_mla_decode)
        assert api.dsa_get_device_error() == 0
        pick = list(range(0, 1024, 41)) + [1023]
        _check({**case, "q": q[pick], "keys": [keys[i] for i in pick], "lens": [lens[i] for i in pick]},
               out[pick], lse[pick], 2.0 ** -8 if fp8 else 0.0)


@pytest.mark.gpu
def test_binding_checks(L):
    c = _case([100, 50], 1, 16, seed=6)
    ws = torch.empty(api.dsa_mla_decode_workspace_bytes(c["desc"]), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 16, 512), dtype=torch.bfloat16, device="cuda")
    call = lambda q=c["q"], kv=c["kv"], out=out, ws=ws, **k: api.dsa_mla_decode(c["desc"], q, kv, out, ws, SM, **k)
    call()
    with pytest.raises(ValueError, match="q:"):
        call(q=c["q"][:1])
    with pytest.raises(ValueError, match="kv:"):
        call(kv=c["kv"][:64])
    with pytest.raises(TypeError, match="out:"):
        call(out=out.float())
    with pytest.raises(ValueError, match="lse:"):
        call(lse=torch.empty((2, 8), device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        call(q=c["q"].cpu())
    with pytest.raises(api.DSAError, match="WORKSPACE"):
        call(ws=ws[:-1])
    with pytest.raises(ValueError, match="kv8:"):
        api.dsa_mla_decode_fp8kv(c["desc"], c["q"], torch.empty((64, 656), dtype=torch.uint8, device="cuda"), out, ws, SM)

"""Attention over FP8 rows of a layer with grouped heads, against its formula in float64 over code x scale.

Tolerances, fixed beforehand.  With A = sum_s p_s |v_s|, E the largest sm_scale * sum_d |q_d k_d| of a row's keys and
Q the largest sm_scale * max|q| * sum_d |k_d|: scores are sums of 2 * 128 products in fp32 and two products with
scales (258 * 2^-24 E), of a query that is off by 2^-17 of its largest value where a value is below 2^-9 of it
(2^-17 Q): dx.  A weight is 2^(x + log2(scale) - m): its exponent is off by dx / ln 2, by the logarithm (2^-22 of it)
and by the roundings of the sum (2^-23 of its terms, at most z = |x| / ln 2 + |log2 scale|): 2^-21 z; it is rounded to
fp16 (2^-11).  Up to 16 rows it is then four E5M2 parts, whole multiples of 2^-16 where the largest weight is 2^13 at
least: cut by up to 2^-29 of the largest.  (More rows: fp16's smallest step, 2^-24, where the largest is 2^7: 2^-32, half
a step.)  So out is off by 2^-8 |out| + (2^-11 + 2.1 (dx + 2^-21 z) + n 2^-24 + 2^-18) A + n 2^-29 max|v|, and the
log-sum-exp by dx + 2^-21 z + n 2^-24 + 2^-20 + 2^-23 |lse|.
"""
import math

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from test_gqa_decode import CASES, FAKE, INF, _desc

D = 128


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_refusals_on_the_host(L):
    def call(desc, **over):
        a = dict(kv=4, dim=128, q=FAKE, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE,
                 ws_bytes=1 << 30)
        return L.dsa_gqa_decode_fp8kv(desc, *{**a, **over}.values(), None)

    for bad in (dict(kv=0), dict(kv=5), dict(q=None), dict(k=None), dict(ks=None), dict(v=None), dict(vs=None), dict(out=None),
                dict(k=FAKE + 8), dict(v=FAKE + 4), dict(ks=FAKE + 4), dict(vs=FAKE + 8), dict(scale=-1.0)):
        assert call(_desc(), **bad) == 1, bad
    for bad in (dict(dim=64), dict(dim=96), dict(dim=256)):
        assert call(_desc(), **bad) == 2, bad
    assert call(_desc(), ws=None) == 3 and call(_desc(batch=0)) == 1 and call(_desc(batch=2000)) == 2


def _case(lens, nq, H, K, seed, spread=4, extra_pages=3, max_pages=None):
    """Codes and scales (powers of two over 2 * spread binades times 1 to 2) in pages of random order; NaN codes and
    scales behind a request's end and in spare pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = [-(-n // 64) for n in lens]
    num_pages = sum(pages) + extra_pages
    max_pages = max_pages or max(1, max(pages))
    ids = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    codes = [torch.full((num_pages, K, 64, D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((num_pages, K, 64), float("nan"), device="cuda") for _ in range(2)]
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = ids[at:at + n]
        at += n
        for i in range(2):
            rows = torch.full((n * 64, K, D), 0x7f, dtype=torch.uint8, device="cuda")
            x = (torch.randn(lens[r], K, D, generator=g, device="cuda") * 120).clamp(-448, 448)      # (beyond: NaN)
            rows[:lens[r]] = x.to(torch.float8_e4m3fn).view(torch.uint8)
            sc = torch.full((n * 64, K), float("nan"), device="cuda")
            w = spread if i else min(spread, 1)
            exp = torch.randint(-w, w + 1, (lens[r], K), generator=g, device="cuda").float()
            sc[:lens[r]] = (1 + torch.rand(lens[r], K, generator=g, device="cuda")) * torch.exp2(exp - 8)
            where = table[r, :n].long().cuda()
            codes[i][where] = rows.unflatten(0, (n, 64)).transpose(1, 2)
            scales[i][where] = sc.unflatten(0, (n, 64)).transpose(1, 2)
    q = torch.randn(len(lens) * nq, H, D, generator=g, device="cuda")
    q *= torch.exp2(torch.randint(-12, 1, q.shape, generator=g, device="cuda").float())      # values far below a row's largest
    q = q.to(torch.bfloat16)
    seq, table = torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()
    desc = api.make_desc(seq, table, nq, H, 1, num_pages)
    ws = torch.full((api.dsa_gqa_decode_workspace_bytes(desc, K, D),), 255, dtype=torch.uint8, device="cuda")
    return dict(desc=desc, q=q, k=codes[0], v=codes[1], ks=scales[0], vs=scales[1], seq=seq, table=table, lens=lens, nq=nq,
                H=H, K=K, ws=ws)


def _run(c, lse=True, stream=None, out=None):
    T = len(c["lens"]) * c["nq"]
    if out is None:
        out = torch.full((T, c["H"], D), 77.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full((T, c["H"]), 77.0, device="cuda") if lse else None
    api.dsa_gqa_decode_fp8kv(c["desc"], c["q"], c["k"], c["ks"], c["v"], c["vs"], out, c["ws"], D ** -0.5, lse=e, stream=stream)
    return out, e


def _check(c, out, lse, heads=None, keys=None):
    nq, G = c["nq"], c["H"] // c["K"]
    sm = D ** -0.5
    for r, n in enumerate(c["lens"]):
        at = c["table"][r, :-(-n // 64)].long()
        for h in heads if heads is not None else range(c["H"]):
            kv = []
            for x, s in (("k", "ks"), ("v", "vs")):
                code = c[x][at, h // G].flatten(0, 1)[:n].view(torch.float8_e4m3fn).double()
                kv.append(code * c[s][at, h // G].flatten()[:n, None].double())
            k, v = kv
            q = c["q"][r * nq:(r + 1) * nq, h].double()
            lim = (n - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0)
            hide = torch.arange(n, device="cuda")[None, :] >= lim[:, None]
            if keys is not None:
                hide = hide | ~keys(r)[None, :]
            empty = hide.all(dim=1) if n else torch.ones(nq, dtype=torch.bool, device="cuda")
            got, e_got = out[r * nq:(r + 1) * nq, h].double(), None if lse is None else lse[r * nq:(r + 1) * nq, h].double()
            assert (got[empty] == 0).all()
            if lse is not None:
                assert (e_got[empty] == -INF).all()
            if bool(empty.all()):
                continue
            x = (sm * (q @ k.T)).masked_fill(hide, -INF)[~empty]
            E = (sm * (q.abs() @ k.abs().T)).masked_fill(hide, 0.0)[~empty].amax(1)
            Q = (sm * q.abs().amax(1)[:, None] * k.abs().sum(1)[None, :]).masked_fill(hide, 0.0)[~empty].amax(1)
            lg = torch.log2(c["vs"][at, h // G].flatten()[:n].double()).abs()
            z = (x.abs().masked_fill(x.isinf(), 0.0) / math.log(2) + lg[None, :]).masked_fill(hide[~empty], 0.0).amax(1)
            got = got[~empty]
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            v = torch.where((~hide).any(0)[:, None], v, 0.0)
            dx = 258 * 2.0 ** -24 * E + 2.0 ** -17 * Q + 2.0 ** -21 * z
            ref, A = p @ v, p @ v.abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.1 * dx[:, None] + n * 2.0 ** -24 + 2.0 ** -18) * A \
                + n * 2.0 ** -29 * v.abs().amax()
            assert ((got - ref).abs() <= tol).all(), (r, n, h, ((got - ref).abs() / tol).max())
            if lse is not None:
                bound = dx + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * e.abs()
                assert ((e_got[~empty] - e).abs() <= bound).all(), (r, n, h)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nq,H,K", CASES)
def test_matches_formula(L, lens, nq, H, K):
    c = _case(lens, nq, H, K, seed=sum(lens) + nq * 7 + H)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=range(0, H, max(1, H // 10)))
    again, _ = _run(c, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
def test_many_requests(L):
    g = torch.Generator().manual_seed(4)
    lens = [int(x) for x in torch.randint(0, 700, (1024,), generator=g)]
    c = _case(lens, 1, 8, 2, seed=1)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=[0, 7])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nq,H,K", [([3000, 1111], 1, 8, 2), ([6000], 3, 20, 1), ([2500] * 5, 2, 96, 2)])
def test_scales_over_many_powers_of_two(L, lens, nq, H, K):
    """Value scales over eighty binades: a weight's exponent takes them, fp16 never sees them."""
    c = _case(lens, nq, H, K, seed=sum(lens) + H, spread=40)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=range(0, H, max(1, H // 5)))


@pytest.mark.gpu
@pytest.mark.parametrize("ramp", ["rise", "fall"])
def test_scores_over_many_powers_of_two(L, ramp):
    """Key scales that rise or fall along the request, on scores that are all positive or negative: the running
    maximum rises again and again, or the tail is lost."""
    lens = [3000, 700, 129]
    c = _case(lens, 2, 12, 2, seed=9)
    c["q"].copy_(c["q"].abs())
    for r, n in enumerate(lens):
        at = c["table"][r, :-(-n // 64)].long()
        t = torch.arange(at.shape[0] * 64, dtype=torch.float32, device="cuda")
        t = 2.0 ** -9 * (1 + (t if ramp == "rise" else t.max() - t) / 100)
        t[n:] = float("nan")
        c["ks"][at] = t.view(-1, 1, 64)
        c["k"][at] = torch.where(c["k"][at] == 0x7f, 0x7f, c["k"][at] & 0x7f)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse)


@pytest.mark.gpu
def test_a_peak_and_a_long_tail(L):
    """One key far above many thousands of equal ones that together weigh as much: no weight may be lost."""
    n = 30000
    c = _case([n], 1, 8, 1, seed=2, spread=0)
    at = c["table"][0].long()
    c["k"][at] = 0
    c["k"][at[0], 0, 0] = 0x38                      # ones
    c["ks"].fill_(2.0 ** -3)
    c["q"].fill_(math.log(n) * D ** 0.5 / D * 8)    # the first key's score: log n
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse)
    assert (lse - math.log(2 * n)).abs().max() < 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("H,K", [(8, 2), (48, 2)])
def test_tiny_value_scales(L, H, K):
    """Value scales below 2^-80, down to 0, count as 2^-80, among others and alone, over many tokens: sums of weights
    over them stay finite."""
    c = _case([500, 300, 70000], 1, H, K, seed=4, spread=2)
    for r, scales in enumerate(([0.0, 2.0 ** -130, 2.0 ** -90, 2.0 ** -8], [2.0 ** -140, 2.0 ** -79], [2.0 ** -100])):
        at = c["table"][r, :-(-c["lens"][r] // 64)].long()
        rows = c["vs"][at].transpose(1, 2).reshape(-1, K)
        rows[:c["lens"][r]] = torch.tensor(scales, device="cuda")[torch.arange(c["lens"][r], device="cuda") % len(scales)][:, None]
        c["vs"][at] = rows.view(len(at), 64, K).transpose(1, 2)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(dict(c, vs=c["vs"].clamp(min=2.0 ** -80)), out, lse, heads=(0, H - 1))


@pytest.mark.gpu
def test_rows_of_tiny_values_as_written(L):
    """What dsa_kv_write_fp8 makes of rows down to the smallest bf16 values can be read."""
    n, K, H = 130, 2, 8
    x = [torch.randn(n, K, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)) for i in (5, 6)]
    x[1] *= torch.tensor([2.0 ** -120, 2.0 ** -70, 1.0, 0.0, 2.0 ** -131], device="cuda")[torch.arange(n, device="cuda") % 5][:, None, None]
    k, v = (t.to(torch.bfloat16) for t in x)
    c = _case([n], 1, H, K, seed=7)
    table = c["table"][0].long()
    slots = (table[torch.arange(n, device="cuda") // 64] * 64 + torch.arange(n, device="cuda") % 64).to(torch.int32)
    api.dsa_kv_write_fp8(k, v, slots, c["k"], c["ks"], c["v"], c["vs"])
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(dict(c, vs=c["vs"].clamp(min=2.0 ** -80)), out, lse)


@pytest.mark.gpu
def test_bad_pages_streams_and_graph(L):
    c = _case([700, 300, 64, 500], 1, 8, 2, seed=3, max_pages=11)
    good, e_good = _run(c)
    assert api.dsa_get_device_error() == 0
    saved = c["table"].clone()
    for bad in (c["desc"].num_pages, -2 ** 31):
        c["table"][0, 4], c["table"][3, 0] = bad, bad
        out, lse = _run(c)
        assert api.dsa_get_device_error() == 5
        c["table"].copy_(saved)
        hidden = {0: 4, 3: 0}
        _check(c, out, lse, keys=lambda r: torch.arange(c["lens"][r], device="cuda") // 64 != hidden.get(r, -1))
        assert torch.equal(out[1:3], good[1:3])
    d = _case([5000, 40], 3, 40, 8, seed=5)
    want = _run(d)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, x in zip(streams, (c, d)):
            with torch.cuda.stream(s):
                got.append(_run(x, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, good) for x in got[::2]) and all(torch.equal(x, want) for x in got[1::2])
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(d, lse=False, out=out)
    graph.replay()
    assert torch.equal(out, want)
    d["seq"].copy_(torch.tensor([129, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _check({**d, "lens": [129, 0]}, out, None)
    assert api.dsa_get_device_error() == 0


@pytest.mark.gpu
def test_binding_checks(L):
    c = _case([100], 1, 8, 2, seed=7)
    _run(c)
    with pytest.raises(ValueError, match="k_scale:"):
        _run({**c, "ks": c["ks"][:, :1]})
    with pytest.raises(ValueError, match="v8:"):
        _run({**c, "v": c["v"][:1]})
    with pytest.raises(TypeError, match="k8:"):
        _run({**c, "k": c["k"].view(torch.float8_e4m3fn)})
    with pytest.raises(TypeError, match="v_scale:"):
        _run({**c, "vs": c["vs"].double()})

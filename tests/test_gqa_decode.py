"""Attention over the paged cache of a layer with grouped heads, against its formula in float64.

Tolerances, fixed beforehand, as for dense latent attention: with A = sum_s p_s |v_s| and E the largest sm_scale *
sum_d |q_d k_d| of a row's keys, scores are off by dx = D * 2^-24 * E, the output by 2^-8 |out| + (2^-8 + 2.1 dx +
n 2^-24 + 2^-18) A, the log-sum-exp by dx + n 2^-24 + 2^-20 + 2^-23 |lse|.
"""
import math

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

FAKE = 0x7f0000000000
INF = float("inf")


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _desc(**over):
    a = dict(batch=2, q_per_req=1, num_heads=16, topk=1, page_size=64, max_pages=3, num_pages=6, seqlens=FAKE,
             page_table=FAKE)
    return api.DecodeDesc(**{**a, **over})


def _raw(L, desc, **over):
    a = dict(kv=4, dim=128, q=FAKE, k=FAKE, v=FAKE, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 30)
    return L.dsa_gqa_decode(desc, *{**a, **over}.values(), None)


def test_refusals_on_the_host(L):
    assert _raw(L, None) == 1
    for bad in (dict(kv=0), dict(kv=5), dict(kv=32), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=FAKE + 8),
                dict(k=FAKE + 8), dict(v=FAKE + 4), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=INF)):
        assert _raw(L, _desc(), **bad) == 1, bad
    for bad in (dict(dim=96), dict(dim=256), dict(dim=576)):
        assert _raw(L, _desc(), **bad) == 2, bad
    for bad in (dict(batch=0), dict(q_per_req=0), dict(num_heads=0), dict(seqlens=None), dict(page_table=FAKE + 1)):
        assert _raw(L, _desc(**bad)) == 1, bad
    for bad in (dict(batch=1025), dict(q_per_req=5), dict(num_heads=132), dict(page_size=32), dict(num_pages=1 << 25)):
        assert _raw(L, _desc(**bad)) == 2, bad
    need = L.dsa_gqa_decode_workspace_bytes(_desc(), 4, 128)
    assert need > 0 and L.dsa_gqa_decode_workspace_bytes(_desc(), 5, 128) == 0
    assert L.dsa_gqa_decode_workspace_bytes(_desc(), 4, 96) == 0 and L.dsa_gqa_decode_workspace_bytes(None, 4, 64) == 0
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert _raw(L, _desc(), **bad) == 3, bad


def _case(lens, nq, H, K, D, seed, extra_pages=3, max_pages=None):
    """Pages in random order; rows behind a request's end, spare pages and the entries behind a request's last
    page are NaN or no page."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = [-(-n // 64) for n in lens]
    num_pages = sum(pages) + extra_pages
    max_pages = max_pages or max(1, max(pages))
    ids = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    caches = [torch.full((num_pages, K, 64, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = ids[at:at + n]
        at += n
        for c in caches:
            rows = torch.full((n * 64, K, D), float("nan"), device="cuda")
            rows[:lens[r]] = torch.randn(lens[r], K, D, generator=g, device="cuda")
            c[table[r, :n].long().cuda()] = rows.to(torch.bfloat16).unflatten(0, (n, 64)).transpose(1, 2)
    q = torch.randn(len(lens) * nq, H, D, generator=g, device="cuda").to(torch.bfloat16)
    seq, table = torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()
    desc = api.make_desc(seq, table, nq, H, 1, num_pages)
    ws = torch.full((api.dsa_gqa_decode_workspace_bytes(desc, K, D),), 255, dtype=torch.uint8, device="cuda")
    return dict(desc=desc, q=q, k=caches[0], v=caches[1], seq=seq, table=table, lens=lens, nq=nq, H=H, K=K, D=D, ws=ws)


def _run(c, lse=True, stream=None, ws=None):
    T = len(c["lens"]) * c["nq"]
    out = torch.full((T, c["H"], c["D"]), 77.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full((T, c["H"]), 77.0, device="cuda") if lse else None
    api.dsa_gqa_decode(c["desc"], c["q"], c["k"], c["v"], out, c["ws"] if ws is None else ws, c["D"] ** -0.5, lse=e,
                       stream=stream)
    return out, e


def rows_of(c, cache, r, h, n):
    """The first n rows of request r and key head h."""
    return cache[c["table"][r, :-(-n // 64)].long(), h].flatten(0, 1)[:n]


def _check(c, out, lse, heads=None, keys=None):
    nq, G, D = c["nq"], c["H"] // c["K"], c["D"]
    sm = D ** -0.5
    for r, n in enumerate(c["lens"]):
        for h in heads if heads is not None else range(c["H"]):
            k, v = (rows_of(c, c[x], r, h // G, n).double() for x in "kv")
            q = c["q"][r * nq:(r + 1) * nq, h].double()
            lim = (n - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0)
            hide = torch.arange(n, device="cuda")[None, :] >= lim[:, None]
            if keys is not None:
                hide = hide | ~keys(r)[None, :]
            got, e_got = out[r * nq:(r + 1) * nq, h].double(), None if lse is None else lse[r * nq:(r + 1) * nq, h].double()
            empty = hide.all(dim=1) if n else torch.ones(nq, dtype=torch.bool, device="cuda")
            assert (got[empty] == 0).all()
            if lse is not None:
                assert (e_got[empty] == -INF).all()
            if bool(empty.all()):
                continue
            x = (sm * (q @ k.T)).masked_fill(hide, -INF)[~empty]
            E = (sm * (q.abs() @ k.abs().T)).masked_fill(hide, 0.0)[~empty]
            got = got[~empty]
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            v = torch.where(p.amax(0)[:, None] > 0, v, 0.0)
            dx = D * 2.0 ** -24 * E.amax(1)
            ref, A = p @ v, p @ v.abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.1 * dx[:, None] + n * 2.0 ** -24 + 2.0 ** -18) * A
            assert ((got - ref).abs() <= tol).all(), (r, n, h, ((got - ref).abs() / tol).max())
            if lse is not None:
                bound = dx + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * e.abs()
                assert ((e_got[~empty] - e).abs() <= bound).all(), (r, n, h)


CASES = [
    ([1], 1, 1, 1), ([1], 2, 4, 2), ([64], 1, 8, 1), ([65, 63, 128, 129], 1, 8, 2), ([0, 5, 0, 0, 300], 1, 4, 4),
    ([2, 3, 4, 200], 4, 16, 2), ([4000], 1, 32, 8), ([4000], 1, 32, 1), ([4000], 2, 48, 1), ([900, 12], 4, 48, 1),
    ([777], 1, 128, 1), ([1000, 1], 3, 128, 1), ([700, 300, 64], 2, 33, 1), ([130] * 40, 1, 10, 2), ([1000, 3] * 9, 2, 40, 8),
    ([20000], 1, 8, 8), ([5000, 100, 9000], 3, 24, 4), ([257], 4, 7, 7), ([600] * 3, 3, 35, 5), ([511, 513], 2, 64, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,nq,H,K", CASES)
def test_matches_formula(L, lens, nq, H, K, D):
    c = _case(lens, nq, H, K, D, seed=sum(lens) + nq * 7 + H)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=range(0, H, max(1, H // 10)))
    again, _ = _run(c, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_requests(L, D):
    g = torch.Generator().manual_seed(4)
    lens = [int(x) for x in torch.randint(0, 700, (1024,), generator=g)]
    c = _case(lens, 1, 8, 2, D, seed=1)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=[0, 7])


# Scores that a key's position adds through the last dim: rising by ten powers of two a tile, falling, in waves.
RAMPS = {
    "rise": lambda t: t * (10 * math.log(2) / 128),
    "fall": lambda t: -t * (10 * math.log(2) / 128),
    "waves": lambda t: t * (3 * math.log(2) / 128) + 25 * torch.sin(t / 90),
}


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("lens,nq,H,K", [([3000, 1111], 1, 8, 2), ([6000], 3, 20, 1), ([2500] * 5, 2, 96, 2)])
def test_scores_over_many_powers_of_two(L, lens, nq, H, K, ramp, D):
    c = _case(lens, nq, H, K, D, seed=sum(lens) + H)
    step = 16.0
    c["q"][:, :, -1] = step
    for r, n in enumerate(lens):
        t = torch.arange(-(-n // 64) * 64, dtype=torch.float32, device="cuda")
        t[n:] = float("nan")
        add = (RAMPS[ramp](t) / (step * D ** -0.5)).to(torch.bfloat16).view(-1, 1, 64)
        c["k"][c["table"][r, :-(-n // 64)].long(), :, :, -1] = add
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse, heads=range(0, H, max(1, H // 5)))


@pytest.mark.gpu
def test_bad_pages_and_lengths(L):
    c = _case([700, 300, 64, 500], 1, 8, 2, 128, seed=3, max_pages=11)
    good, _ = _run(c)
    assert api.dsa_get_device_error() == 0
    for bad in (c["desc"].num_pages, 2 ** 31 - 1, -1, -2 ** 31):
        saved = c["table"].clone()
        c["table"][0, 4], c["table"][3, 0] = bad, bad
        out, lse = _run(c)
        assert api.dsa_get_device_error() == 5
        hidden = {0: 4, 3: 0}
        c["table"].copy_(saved)
        keys = lambda r: torch.arange(c["lens"][r], device="cuda") // 64 != hidden.get(r, -1)
        _check(c, out, lse, keys=keys)
        assert torch.equal(out[1:3], good[1:3])
    # a length past the table is cut to it, a negative one counts as none
    c["seq"][0], c["seq"][2] = 11 * 64 + 1, -5
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 5
    assert (out[2] == 0).all() and (lse[2] == -INF).all() and torch.equal(out[1], good[1])
    c["seq"][0] = 700
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0 and torch.equal(out[0], good[0])


@pytest.mark.gpu
def test_streams_graphs_and_workspaces(L):
    c, d = _case([3000, 40], 1, 32, 8, 128, seed=5), _case([900] * 6, 2, 16, 4, 64, seed=6)
    want_c, want_d = _run(c)[0], _run(d)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, x in zip(streams, (c, d)):
            with torch.cuda.stream(s):
                got.append(_run(x, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want_c) for x in got[::2]) and all(torch.equal(x, want_d) for x in got[1::2])
    # two captured steps that share a workspace, replayed in turn, and lengths that change between replays
    ws = torch.empty(max(c["ws"].numel(), d["ws"].numel()), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for x in (c, d):
        out = torch.empty_like(_run(x)[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.dsa_gqa_decode(x["desc"], x["q"], x["k"], x["v"], out, ws, x["D"] ** -0.5)
        outs.append(out)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    assert torch.equal(outs[0], want_c) and torch.equal(outs[1], want_d)
    c["seq"].copy_(torch.tensor([1500, 0], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    _check({**c, "lens": [1500, 0]}, outs[0], None)
    assert api.dsa_get_device_error() == 0


@pytest.mark.gpu
def test_pages_past_two_to_the_31(L):
    """Pages behind 2^31 values of the cache, and rows past 2^31."""
    K, D, pages = 16, 128, 40000
    k, v = (torch.empty((pages, K, 64, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 300
    for x in (k, v):
        x[-5:] = torch.randn(5, K, 64, D, device="cuda").to(torch.bfloat16)
    table = torch.arange(pages - 1, pages - 6, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 32, D, device="cuda").to(torch.bfloat16)
    desc = api.make_desc(seq, table, 1, 32, 1, pages)
    ws = torch.empty(api.dsa_gqa_decode_workspace_bytes(desc, K, D), dtype=torch.uint8, device="cuda")
    c = dict(desc=desc, q=q, k=k, v=v, seq=seq, table=table, lens=[n], nq=1, H=32, K=K, D=D, ws=ws)
    out, lse = _run(c)
    assert api.dsa_get_device_error() == 0
    _check(c, out, lse)


@pytest.mark.gpu
def test_binding_checks(L):
    c = _case([100], 1, 8, 2, 128, seed=7)
    out = torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda q=c["q"], k=c["k"], v=c["v"], out=out, ws=c["ws"], **kw: api.dsa_gqa_decode(c["desc"], q, k, v, out, ws, 0.1, **kw)
    call()
    with pytest.raises(ValueError, match="q:"):
        call(q=c["q"][:, :4])
    with pytest.raises(ValueError, match="v:"):
        call(v=c["v"][:, :1])
    with pytest.raises(ValueError, match="k:"):
        call(k=c["k"][:1])
    with pytest.raises(TypeError, match="k: expected a 4-D"):
        call(k=c["k"][0])
    with pytest.raises(TypeError, match="v:"):
        call(v=c["v"].float())
    with pytest.raises(ValueError, match="out:"):
        call(out=out[..., :64])
    with pytest.raises(TypeError, match="ws:"):
        call(ws=c["ws"].float())
    with pytest.raises(api.DSAError, match="WORKSPACE"):
        call(ws=c["ws"][:256])
    with pytest.raises(api.DSAError, match="INVALID"):
        k = c["k"][:, :1].expand(-1, 3, -1, -1).contiguous()
        call(k=k, v=k)

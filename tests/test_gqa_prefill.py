"""Attention of packed prompts with grouped heads, against its formula in float64.

Tolerances, fixed beforehand, as for prompt attention in the expanded form: with A = sum_j p_j |v_j| and E the
largest sm_scale * sum_d |q_d k_d| of a row's keys, scores are off by dx = D * 2^-24 * E, the output by 2^-8 |out|
+ (2^-8 + 2.1 dx + n 2^-24 + 2^-18) A, the log-sum-exp by dx + n 2^-24 + 2^-20 + 2^-23 |lse|.
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


def _raw(L, **over):
    a = dict(batch=2, heads=16, kv=4, dim=128, tq=64, tk=64, mq=40, cu_q=FAKE, cu_k=FAKE, q=FAKE, ld_q=2048, k=FAKE,
             ld_k=512, v=FAKE, ld_v=512, scale=0.1, causal=1, out=FAKE, lse=FAKE)
    return L.dsa_gqa_prefill(*{**a, **over}.values(), None)


def test_refusals_on_the_host(L):
    assert _raw(L, tq=0) == 0 and _raw(L, mq=0) == 0                 # nothing to do
    for bad in (dict(batch=0), dict(heads=0), dict(kv=0), dict(kv=5), dict(tq=-1), dict(tk=-1), dict(mq=-1),
                dict(ld_q=2040), dict(ld_q=2050), dict(ld_k=504), dict(ld_k=516), dict(ld_v=500), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=INF), dict(cu_q=None), dict(cu_k=None), dict(cu_q=FAKE + 2),
                dict(cu_k=FAKE + 1), dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(q=FAKE + 8),
                dict(k=FAKE + 8), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2)):
        assert _raw(L, **bad) == 1, bad
    for bad in (dict(batch=65536), dict(heads=1028, ld_q=2 ** 18), dict(dim=96), dict(dim=256, ld_q=4096),
                dict(heads=129, kv=1, ld_q=129 * 128), dict(batch=1, heads=1024, kv=1024, dim=64, tq=2 ** 31 - 1, ld_q=65536,
                                                           ld_k=65536, ld_v=65536)):
        assert _raw(L, **bad) == 2, bad


def _case(qlens, klens, H, K, D, seed, fused=False, tail=5):
    """Packed requests; `tail` rows of NaN follow the last one.  fused: queries, keys and values are columns of
    one projection (where there are as many of each)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = lambda n: torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")
    Tq, Tk = sum(qlens), sum(klens)
    if fused:
        rows = torch.cat([rnd(Tq, (H + 2 * K) * D + 8), nan(tail, (H + 2 * K) * D + 8)])
        q, k, v = (x.unflatten(1, (-1, D)) for x in rows[:, 8:].split([H * D, K * D, K * D], dim=1))
    else:
        q, k, v = (torch.cat([rnd(n, h, D), nan(tail, h, D)]) for n, h in ((Tq, H), (Tk, K), (Tk, K)))
    return dict(q=q, k=k, v=v, cu_q=cu(qlens), cu_k=cu(klens), qlens=qlens, klens=klens, H=H, K=K, D=D, max_q=max(qlens))


def _run(c, causal, lse=True, stream=None, out=None):
    if out is None:
        out = torch.full((c["q"].shape[0], c["H"], c["D"]), 77.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full(out.shape[:2], 77.0, device="cuda") if lse else None
    api.dsa_gqa_prefill(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], out, c["max_q"], c["D"] ** -0.5, causal=causal,
                        lse=e, stream=stream)
    return out, e


def _check(c, causal, out, lse, heads=None):
    a = b = 0
    D, G = c["D"], c["H"] // c["K"]
    sm = D ** -0.5
    for n, m in zip(c["qlens"], c["klens"]):
        for h in heads if heads is not None else range(c["H"]):
            q, k, v = c["q"][a:a + n, h].double(), c["k"][b:b + m, h // G].double(), c["v"][b:b + m, h // G].double()
            lim = (torch.arange(n, device="cuda") + (m - n + 1)).clamp(min=0) if causal else torch.full((n,), m, device="cuda")
            hide = torch.arange(m, device="cuda")[None, :] >= lim[:, None]
            x = (sm * (q @ k.T)).masked_fill(hide, -INF)
            E = (sm * (q.abs() @ k.abs().T)).masked_fill(hide, 0.0)
            empty = lim == 0
            got, e_got = out[a:a + n, h].double(), None if lse is None else lse[a:a + n, h].double()
            assert (got[empty] == 0).all()
            if lse is not None:
                assert (e_got[empty] == -INF).all()
            if bool(empty.all()):
                continue
            x, E, got = x[~empty], E[~empty], got[~empty]
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            dx = D * 2.0 ** -24 * E.amax(1)
            ref, A = p @ v, p @ v.abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.1 * dx[:, None] + m * 2.0 ** -24 + 2.0 ** -18) * A
            assert ((got - ref).abs() <= tol).all(), (n, m, h, ((got - ref).abs() / tol).max())
            if lse is not None:
                bound = dx + m * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * e.abs()
                assert ((e_got[~empty] - e).abs() <= bound).all(), (n, m, h)
        a, b = a + n, b + m
    assert (out[a:] == 77).all()                       # rows behind the last request
    assert lse is None or (lse[a:] == 77).all()


CASES = [
    ([1], [1], 1, 1), ([1], [300], 6, 2), ([5], [3], 8, 1), ([4], [0], 4, 2), ([0, 7, 0], [0, 7, 5], 10, 2),
    ([127, 128, 129], [127, 128, 129], 4, 4), ([31, 32, 33], [31, 32, 33], 16, 2), ([15, 16, 17], [140, 16, 129], 32, 4),
    ([255, 256, 257], [255, 256, 257], 2, 1), ([1, 2, 3, 64], [65, 130, 3, 64], 5, 1), ([300], [1000], 14, 2),
    ([513, 40], [700, 41], 24, 8), ([200, 150], [100, 150], 12, 1), ([1000], [1000], 6, 3), ([33] * 20, [33] * 20, 28, 4),
    ([700], [2500], 3, 1), ([3, 2], [300, 2], 128, 1), ([5, 9], [5, 200], 96, 1), ([6], [500], 65, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qlens,klens,H,K", CASES)
def test_matches_formula(L, qlens, klens, H, K, causal, D):
    c = _case(qlens, klens, H, K, D, seed=sum(qlens) * 7 + sum(klens) + H, fused=qlens == klens)
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse, heads=range(0, H, max(1, H // 12)))
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)


# Few items with many keys: the CTAs of a cluster share an item's keys.  More key heads or blocks leave fewer CTAs
# for an item; the last ones have a request with fewer key tiles than there are parts, one or none.
SHARED = [
    ([130], [4100], 8, 8), ([1], [4001], 128, 16), ([40], [3000], 32, 4), ([3], [5000], 24, 24), ([100], [4100], 32, 32),
    ([20], [2500], 80, 40), ([64], [2600], 70, 70), ([2, 200, 2], [9000, 300, 1], 9, 3), ([2, 2, 0], [9000, 0, 5], 20, 4),
    ([300, 5], [6000, 2], 2, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qlens,klens,H,K", SHARED)
def test_shared_keys(L, qlens, klens, H, K, causal, D):
    c = _case(qlens, klens, H, K, D, seed=sum(qlens) * 5 + sum(klens) + H)
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse, heads=range(0, H, max(1, H // 8)))
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)


# Scores (natural logarithms) that a key's position adds through the last dim: rising by ten powers of two a
# 128-key tile, falling as fast, and rising in waves.
RAMPS = {
    "rise": lambda t: t * (10 * math.log(2) / 128),
    "fall": lambda t: -t * (10 * math.log(2) / 128),
    "waves": lambda t: t * (3 * math.log(2) / 128) + 25 * torch.sin(t / 90),
}


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m,H,K", [(1300, 5400, 64, 8), (2700, 6000, 16, 1), (1235, 3001, 40, 8), (2600, 1900, 64, 8)])
def test_a_last_round_that_shares_keys(L, n, m, H, K, causal, D):
    """One request of a few more blocks than there are SMs (or twice as many): all of them are done, once."""
    c = _case([n], [m], H, K, D, seed=n + m)
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse, heads=range(0, H, max(1, H // 5)))
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("qlens,klens,H,K", [([1500, 700], [1500, 2500], 6, 2), ([130], [4100], 8, 8), ([300] * 8, [900] * 8, 40, 8)])
def test_scores_over_many_powers_of_two(L, qlens, klens, H, K, ramp, D):
    c = _case(qlens, klens, H, K, D, seed=sum(qlens) * 3 + sum(klens) + H)
    step = 16.0
    c["q"][:sum(qlens), :, -1] = step
    at = 0
    for m in klens:
        t = torch.arange(m, dtype=torch.float32, device="cuda")
        c["k"][at:at + m, :, -1] = (RAMPS[ramp](t) / (step * D ** -0.5)).to(torch.bfloat16)[:, None]
        at += m
    for causal in (True, False):
        out, lse = _run(c, causal)
        assert api.dsa_get_device_error() == 0
        _check(c, causal, out, lse, heads=range(0, H, max(1, H // 4)))


@pytest.mark.gpu
def test_many_short_requests_and_a_long_one(L):
    qlens = [(i * 7) % 5 for i in range(700)]
    qlens[333] = 1900
    klens = [n + (i % 3) * 50 for i, n in enumerate(qlens)]
    c = _case(qlens, klens, 4, 2, 128, seed=10)
    out, lse = _run(c, True)
    assert api.dsa_get_device_error() == 0
    _check(c, True, out, lse, heads=[1, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("qlens,klens,H,K", [([100, 300, 50], [100, 300, 50], 8, 2), ([100, 300, 50], [4100, 4300, 4050], 8, 1)])
def test_bad_offsets_are_reported(L, qlens, klens, H, K):
    c = _case(qlens, klens, H, K, 128, seed=1)
    good, e_good = _run(c, True)
    assert api.dsa_get_device_error() == 0
    over = lambda **k: {**c, **{n: torch.tensor(o, dtype=torch.int32, device="cuda") for n, o in k.items()}}
    b = c["cu_k"].tolist()
    for offsets, kept in (([0, b[1], b[3], 10 ** 6], [(0, 100)]), ([0, b[1], 20, b[3]], [(0, 100)])):
        out, lse = _run(over(cu_k=offsets), True)
        assert api.dsa_get_device_error() == 5
        for x, y in kept:
            assert torch.equal(out[x:y], good[x:y]) and torch.equal(lse[x:y], e_good[x:y])
        assert (out[450:] == 77).all()
    for offsets in ([0, 300, 250, 450], [0, 10 ** 6, 50, 200], [450, 100, 400, 450], [0, 100, -1, 450]):
        out, lse = _run(over(cu_q=offsets), True)
        assert api.dsa_get_device_error() == 5 and (out == 77).all() and (lse == 77).all()
    for offsets, kept in (([0, 100, 400, 10 ** 6], [(0, 400)]), ([-1, 100, 400, 450], [(100, 450)]),
                          ([0, 100, 10 ** 6, 2 ** 31 - 1], [(0, 100)])):
        out, lse = _run(over(cu_q=offsets), True)
        assert api.dsa_get_device_error() == 5
        left = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
        for x, y in kept:
            assert torch.equal(out[x:y], good[x:y]) and torch.equal(lse[x:y], e_good[x:y]), offsets
            left[x:y] = False
        assert (out[left] == 77).all() and (lse[left] == 77).all()
    out, _ = _run({**c, "max_q": 200}, True)
    assert api.dsa_get_device_error() == 5
    assert torch.equal(out[:300], good[:300]) and torch.equal(out[400:450], good[400:450])
    out, _ = _run({**c, "max_q": 5000}, True)
    assert api.dsa_get_device_error() == 0 and torch.equal(out[:450], good[:450])


@pytest.mark.gpu
def test_streams_and_graphs(L):
    c1, c2 = _case([70, 20], [3000, 20], 8, 2, 128, seed=2), _case([300] * 4, [300] * 4, 16, 4, 64, seed=3)
    want1, want2 = _run(c1, True)[0], _run(c2, False)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s, c, causal in ((streams[0], c1, True), (streams[1], c2, False)):
            with torch.cuda.stream(s):
                got.append(_run(c, causal, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(g, want1) for g in got[0::2]) and all(torch.equal(g, want2) for g in got[1::2])
    out = torch.full_like(want1, 77.0)
    q0, cu0 = c1["q"].clone(), c1["cu_q"].clone()
    c1["q"].zero_()
    c1["cu_q"].copy_(torch.tensor([0, 1, 2], dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c1, True, lse=False, out=out)
    c1["q"].copy_(q0)
    c1["cu_q"].copy_(cu0)
    graph.replay()
    assert torch.equal(out, want1) and api.dsa_get_device_error() == 0


@pytest.mark.gpu
def test_keys_past_two_to_the_31(L):
    """The second request's keys lie behind 2^31 values of the packed tensors, and the queries' rows far apart."""
    H, K, D, far = 32, 8, 128, 2100000
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.zeros((far + 300, K, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (k, v):
        x[far:] = torch.randn(300, K, D, generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.empty((151, 1 << 24), dtype=torch.bfloat16, device="cuda")
    q = rows[:, :H * D].unflatten(1, (H, D))
    q.copy_(torch.randn(151, H, D, generator=g, device="cuda"))
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    out = torch.empty((151, H, D), dtype=torch.bfloat16, device="cuda")
    api.dsa_gqa_prefill(q, k, v, cu(0, 1, 151), cu(0, far, far + 300), out, 150, D ** -0.5)
    assert api.dsa_get_device_error() == 0
    assert (out[0] == 0).all()                       # a mean of zero values
    c = dict(q=q[1:], k=k[far:], v=v[far:], qlens=[150], klens=[300], H=H, K=K, D=D)
    _check(c, True, out[1:], None, heads=[0, 17, 31])


@pytest.mark.gpu
def test_an_output_off_32_bytes(L):
    c = _case([130, 40], [300, 40], 6, 2, 64, seed=9)
    want, _ = _run(c, True)
    n = want.numel()
    buf = torch.full((n + 16,), 77.0, dtype=torch.bfloat16, device="cuda")
    for off in (8, 16):
        out = buf[off:off + n].view(want.shape)
        assert out.data_ptr() % 32 == (16 if off == 8 else 0)
        _run(c, True, lse=False, out=out)
        assert torch.equal(out, want) and (buf[:off] == 77).all() and (buf[off + n:] == 77).all()
        buf.fill_(77.0)


@pytest.mark.gpu
def test_binding_checks(L):
    c = _case([20], [20], 4, 2, 128, seed=6, tail=0)
    out = torch.empty((20, 4, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda q=c["q"], k=c["k"], v=c["v"], cu_q=c["cu_q"], cu_k=c["cu_k"], out=out, **kw: \
        api.dsa_gqa_prefill(q, k, v, cu_q, cu_k, out, 20, 0.1, **kw)
    call()
    with pytest.raises(ValueError, match="v:"):
        call(v=c["v"][:, :1])
    with pytest.raises(ValueError, match="k: expected shape"):
        call(q=c["q"][..., :64].contiguous())
    with pytest.raises(ValueError, match="q: expected contiguous heads"):
        call(q=c["q"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(TypeError, match="cu_k:"):
        call(cu_k=c["cu_k"].long())
    with pytest.raises(ValueError, match="cu_k:"):
        call(cu_k=c["cu_k"][:1])
    with pytest.raises(TypeError, match="cu_q"):
        call(cu_q=c["cu_q"][:1])
    with pytest.raises(ValueError, match="out:"):
        call(out=out[:10])
    with pytest.raises(ValueError, match="lse:"):
        call(lse=torch.empty((20, 5), device="cuda"))

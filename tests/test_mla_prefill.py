"""Prompt attention over expanded keys and values, against its formula in float64.

Tolerances, fixed beforehand, as for the dense decode: with A = sum_j p_j |v_j| and E the largest
sm_scale * sum_d |q_d k_d| of a row's keys, scores are off by dx = 192 * 2^-24 * E, the output by
2^-8 |out| + (2^-8 + 2.1 dx + n 2^-24 + 2^-18) A, the log-sum-exp by dx + n 2^-24 + 2^-20 + 2^-23 |lse|.
"""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

SM = 1.0 / 192.0 ** 0.5
FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_refusals_on_the_host(L):
    ok = dict(batch=2, heads=16, tq=64, tk=64, mq=40, cu_q=FAKE, cu_k=FAKE, q=FAKE, kv=FAKE, rope=FAKE,
              ld=576, scale=SM, causal=1, out=FAKE, lse=FAKE)

    def call(**over):
        a = {**ok, **over}
        return L.dsa_mla_prefill(a["batch"], a["heads"], a["tq"], a["tk"], a["mq"], a["cu_q"], a["cu_k"],
                                 a["q"], a["kv"], a["rope"], a["ld"], a["scale"], a["causal"], a["out"],
                                 a["lse"], None)

    assert call(tq=0) == 0 and call(mq=0) == 0                 # nothing to do
    for bad in (dict(batch=0), dict(heads=0), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(ld=56),
                dict(ld=68), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(cu_q=None), dict(cu_k=None), dict(cu_q=FAKE + 2), dict(cu_k=FAKE + 1), dict(q=None),
                dict(out=None), dict(kv=None), dict(rope=None), dict(q=FAKE + 8), dict(kv=FAKE + 8),
                dict(rope=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(batch=65536), dict(heads=1025)):
        assert call(**bad) == 2, bad


def _case(qlens, klens, H, seed, tail=5):
    """Packed requests; `tail` rows of NaN follow the last one, and the rope keys lie in wider rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    cu = lambda n: torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")
    Tq, Tk = sum(qlens), sum(klens)
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.cat([rnd(Tq, H, 192), nan(tail, H, 192)])
    kv = torch.cat([rnd(Tk, H, 256), nan(tail, H, 256)])
    latent = nan(Tk + tail, 576)
    latent[:Tk, 512:] = rnd(Tk, 64)
    return dict(q=q, kv=kv, rope=latent[:, 512:], cu_q=cu(qlens), cu_k=cu(klens), qlens=qlens, klens=klens, H=H,
                max_q=max(qlens))


def _run(c, causal, lse=True, stream=None):
    out = torch.full(c["q"].shape[:2] + (128,), 77.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full(c["q"].shape[:2], 77.0, device="cuda") if lse else None
    api.dsa_mla_prefill(c["q"], c["kv"], c["rope"], c["cu_q"], c["cu_k"], out, c["max_q"], SM, causal=causal,
                        lse=e, stream=stream)
    return out, e


def _check(c, causal, out, lse, heads=None):
    a = b = 0
    for n, m in zip(c["qlens"], c["klens"]):
        for h in heads if heads is not None else range(c["H"]):
            q = c["q"][a:a + n, h].double()
            k = torch.cat([c["kv"][b:b + m, h, :128], c["rope"][b:b + m]], dim=1).double()
            v = c["kv"][b:b + m, h, 128:].double()
            lim = (torch.arange(n, device="cuda") + (m - n + 1)).clamp(min=0) if causal else torch.full((n,), m, device="cuda")
            hide = torch.arange(m, device="cuda")[None, :] >= lim[:, None]
            x = (SM * (q @ k.T)).masked_fill(hide, float("-inf"))
            E = (SM * (q.abs() @ k.abs().T)).masked_fill(hide, 0.0)
            empty = lim == 0
            got, e_got = out[a:a + n, h].double(), None if lse is None else lse[a:a + n, h].double()
            assert (got[empty] == 0).all()
            if lse is not None:
                assert (e_got[empty] == float("-inf")).all()
            if bool(empty.all()):
                continue
            x, E, got = x[~empty], E[~empty], got[~empty]
            e = torch.logsumexp(x, 1)
            p = torch.exp(x - e[:, None])
            dx = 192 * 2.0 ** -24 * E.amax(1)
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
    ([1], [1], 1), ([1], [300], 3), ([5], [3], 2), ([4], [0], 2), ([0, 7, 0], [0, 7, 5], 2),
    ([127, 128, 129], [127, 128, 129], 4), ([255, 256, 257], [255, 256, 257], 3),
    ([1, 2, 3, 64], [65, 130, 3, 64], 5), ([300], [1000], 7), ([513, 40], [700, 41], 8),
    ([200, 150], [100, 150], 2), ([1000], [1000], 2), ([33] * 20, [33] * 20, 2), ([700], [2500], 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qlens,klens,H", CASES)
def test_matches_formula(L, qlens, klens, H, causal):
    c = _case(qlens, klens, H, seed=sum(qlens) * 7 + sum(klens) + H)
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse)
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
def test_bad_offsets_are_reported(L):
    c = _case([100, 300, 50], [100, 300, 50], 4, seed=1)
    good, _ = _run(c, True)
    # the second request's keys would end behind the packed tensor: skipped, the others as before
    saved = c["cu_k"].clone()
    c["cu_k"][2:] += 1000
    out, _ = _run(c, True)
    assert api.dsa_get_device_error() == 5
    assert torch.equal(out[:100], good[:100]) and (out[100:450] == 77).all()
    # ... or come before the first request's
    c["cu_k"].copy_(saved)
    c["cu_k"][2] = 20
    out, _ = _run(c, True)
    assert api.dsa_get_device_error() == 5
    assert torch.equal(out[:100], good[:100]) and (out[100:400] == 77).all()
    c["cu_k"].copy_(saved)
    # a request longer than max_q says (rounded up to 256): its first queries are written
    out, _ = _run({**c, "max_q": 200}, True)
    assert api.dsa_get_device_error() == 5
    assert torch.equal(out[:100], good[:100]) and torch.equal(out[400:450], good[400:450])
    out, _ = _run({**c, "max_q": 5000}, True)
    assert api.dsa_get_device_error() == 0 and torch.equal(out[:450], good[:450])


@pytest.mark.gpu
def test_streams_and_graphs(L):
    c1, c2 = _case([700, 20], [900, 20], 8, seed=2), _case([300] * 4, [300] * 4, 16, seed=3)
    want1, want2 = _run(c1, True)[0], _run(c2, False)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, c, causal in ((s1, c1, True), (s2, c2, False)):
            with torch.cuda.stream(s):
                got.append(_run(c, causal, stream=s)[0])
    torch.cuda.synchronize()
    eq = lambda a, b, n: torch.equal(a[:n], b[:n])
    assert all(eq(g, want1, 720) for g in got[0::2]) and all(eq(g, want2, 1200) for g in got[1::2])
    out = torch.empty_like(want1)
    q0, cu0 = c1["q"].clone(), c1["cu_q"].clone()
    c1["q"].zero_()
    c1["cu_q"].copy_(torch.tensor([0, 1, 2], dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dsa_mla_prefill(c1["q"], c1["kv"], c1["rope"], c1["cu_q"], c1["cu_k"], out, c1["max_q"], SM)
    c1["q"].copy_(q0)
    c1["cu_q"].copy_(cu0)
    graph.replay()
    assert eq(out, want1, 720) and api.dsa_get_device_error() == 0


@pytest.mark.gpu
def test_large_scores_raise_the_maximum(L):
    """Keys that grow along the request: the running maximum rises by far more than 2^8 several times."""
    c = _case([700], [700], 2, seed=5)
    ramp = (1.0 + torch.arange(700, device="cuda") / 40.0).to(torch.bfloat16)
    c["kv"][:700, :, :128] *= ramp[:, None, None]
    out, lse = _run(c, True)
    _check(c, True, out, lse)


@pytest.mark.gpu
def test_keys_past_two_to_the_31(L):
    """The second request's keys lie behind 2^31 values of the packed tensor."""
    H, far = 128, 66000
    g = torch.Generator(device="cuda").manual_seed(8)
    kv = torch.zeros((far + 300, H, 256), dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros((far + 300, 64), dtype=torch.bfloat16, device="cuda")
    kv[far:] = torch.randn(300, H, 256, generator=g, device="cuda").to(torch.bfloat16)
    rope[far:] = torch.randn(300, 64, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1 + 150, H, 192, generator=g, device="cuda").to(torch.bfloat16)
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    out = torch.empty((151, H, 128), dtype=torch.bfloat16, device="cuda")
    api.dsa_mla_prefill(q, kv, rope, cu(0, 1, 151), cu(0, far, far + 300), out, 150, SM)
    assert api.dsa_get_device_error() == 0
    assert (out[0] == 0).all()                       # a mean of zero values
    c = dict(q=q[1:], kv=kv[far:], rope=rope[far:], qlens=[150], klens=[300], H=H)
    _check(c, True, out[1:], None, heads=[0, 77, 127])


@pytest.mark.gpu
def test_binding_checks(L):
    c = _case([20], [20], 4, seed=6, tail=0)
    out = torch.empty((20, 4, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda q=c["q"], kv=c["kv"], rope=c["rope"], cu_q=c["cu_q"], cu_k=c["cu_k"], out=out, **k: \
        api.dsa_mla_prefill(q, kv, rope, cu_q, cu_k, out, 20, SM, **k)
    call()
    call(rope=c["rope"].contiguous())
    with pytest.raises(ValueError, match="kv:"):
        call(kv=c["kv"][:, :2])
    with pytest.raises(ValueError, match="q:"):
        call(q=c["q"][..., :128])
    with pytest.raises(ValueError, match="64 columns"):
        call(rope=c["rope"][:, :32])
    with pytest.raises(ValueError, match="contiguous columns"):
        call(rope=c["rope"].contiguous().t().contiguous().t())
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


@pytest.mark.gpu
def test_an_output_off_32_bytes(L):
    """Outputs are stored 32 bytes at a time where they are aligned so; 16 bytes suffice."""
    c = _case([130, 40], [300, 40], 3, seed=9)
    want, _ = _run(c, True)
    n = want.numel()
    buf = torch.full((n + 16,), 77.0, dtype=torch.bfloat16, device="cuda")
    for off in (8, 16):
        out = buf[off:off + n].view(want.shape)
        assert out.data_ptr() % 32 == (16 if off == 8 else 0)
        api.dsa_mla_prefill(c["q"], c["kv"], c["rope"], c["cu_q"], c["cu_k"], out, c["max_q"], SM)
        assert torch.equal(out[:170], want[:170])
        assert (buf[:off] == 77).all() and (buf[off + n:] == 77).all()
        buf.fill_(77.0)


@pytest.mark.gpu
def test_many_short_requests_and_a_long_one(L):
    qlens = [(i * 7) % 5 for i in range(700)]
    qlens[333] = 1900
    klens = [n + (i % 3) * 50 for i, n in enumerate(qlens)]
    c = _case(qlens, klens, 2, seed=10)
    out, lse = _run(c, True)
    assert api.dsa_get_device_error() == 0
    _check(c, True, out, lse, heads=[1])


# Few items with many keys: the CTAs of a cluster share an item's keys.  More heads leave fewer CTAs for
# an item (8: six to eight, 16: six, 24: five, 32: four, 40: three, 70: two on 152 SMs); the last ones have a request
# with fewer key tiles than there are parts, one or none.
SHARED = [
    ([130], [4100], 8), ([1], [4001], 16), ([257], [3000], 8), ([3], [5000], 24), ([100], [4100], 32),
    ([129], [2500], 40), ([64], [2600], 70), ([2, 200, 2], [9000, 300, 1], 3), ([2, 2, 0], [9000, 0, 5], 4),
    ([300, 5], [6000, 2], 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qlens,klens,H", SHARED)
def test_shared_keys(L, qlens, klens, H, causal):
    c = _case(qlens, klens, H, seed=sum(qlens) * 5 + sum(klens) + H)
    out, lse = _run(c, causal)
    assert api.dsa_get_device_error() == 0
    _check(c, causal, out, lse, heads=range(0, H, max(1, H // 8)))
    again, _ = _run(c, causal, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
def test_shared_keys_bad_offsets_streams_and_graph(L):
    c = _case([70, 100], [4000, 3000], 8, seed=3)
    good, e_good = _run(c, True)
    saved = c["cu_k"].clone()
    c["cu_k"][2] += 1000
    out, _ = _run(c, True)
    assert api.dsa_get_device_error() == 5
    assert torch.equal(out[:70], good[:70]) and (out[70:] == 77).all()
    c["cu_k"].copy_(saved)
    # two calls at once, and a captured one that finds other lengths when it is replayed
    d = _case([33], [6000], 8, seed=4)
    d_good, _ = _run(d, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, x in zip(streams, (c, d)):
            with torch.cuda.stream(s):
                got.append(_run(x, True)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, good) for a in got[::2]) and all(torch.equal(a, d_good) for a in got[1::2])
    out, e = torch.full_like(good, 77.0), torch.full_like(e_good, 77.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.dsa_mla_prefill(c["q"], c["kv"], c["rope"], c["cu_q"], c["cu_k"], out, c["max_q"], SM, lse=e)
    g.replay()
    assert torch.equal(out, good) and torch.equal(e, e_good)
    c["cu_k"].copy_(torch.tensor([0, 5000, 7000], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    _check({**c, "klens": [5000, 2000]}, True, out, e)
    assert api.dsa_get_device_error() == 0

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

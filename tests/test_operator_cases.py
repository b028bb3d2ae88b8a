"""The measured cases of perf/operators.py, and some drawn from their ranges, against their float64 definitions.

Tolerances, as in the tests of each operator: with A = sum p |v| (exact probabilities) and E the largest
sm_scale * sum |q||k| of a row, scores are off by dx = dims * 2^-24 * E, an output by 2^-8 |out| + (2^-8 +
2.1 dx + n 2^-24 + 2^-18) A over n keys, a log-sum-exp by dx + n 2^-24 + 2^-20 + 2^-23 |lse|; FP8 rows count as
they are multiplied (code times scale in fp32, rounded to bf16).  The norm's bf16 outputs are off by 2^-8 of
their value and 2^-17 for the arithmetic, a code times its scale by 2^-4 of the value or 2^-10 of the scale.
"""
import random

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from perf import operators


def test_cases_are_named_once_and_cover_every_operator():
    cases = operators.listed()
    assert len({c["name"] for c in cases}) == len(cases)
    assert {c["op"] for c in cases} == {"decode", "prompt", "norm"} and not operators.own
    for seed in range(200):
        assert all(v > 0 for v in operators.work(operators.draw(random.Random(seed))).values())


def _bounds(q, k, v, limit):
    """In place of an attention's (output, lse): (A, E)."""
    hide = torch.arange(k.shape[0], device=q.device)[None, :] >= limit[:, None]
    x = ((q @ k.T) * operators.SM_SCALE).masked_fill_(hide, float("-inf"))
    size = ((q.abs() @ k.abs().T) * operators.SM_SCALE).masked_fill_(hide, 0.0)
    return torch.softmax(x, dim=1) @ v.abs(), size.amax(dim=1)


def _attention(case, seed, got, monkeypatch):
    attend = operators._attend64
    if case.get("cache") == "fp8":
        mult = lambda t: t.float().to(torch.bfloat16).double()
        attend = lambda q, k, v, limit, inner=attend: inner(q, mult(k), mult(v), limit)
    whole = {**case, "lse": True}
    monkeypatch.setattr(operators, "_attend64", attend)
    want = operators.exact(whole, seed)
    monkeypatch.setattr(operators, "_attend64", _bounds)
    bound = operators.exact(whole, seed)
    A, E = bound["out"], bound["lse"]
    n = case["hi"] if case["op"] == "decode" else case["qhi"] + case["prefix"]
    dx = (576 if case["op"] == "decode" else 192) * 2.0 ** -24 * E
    tol = 2.0 ** -8 * want["out"].abs() + (2.0 ** -8 + 2.1 * dx[..., None] + n * 2.0 ** -24 + 2.0 ** -18) * A
    assert got["out"].dtype == torch.bfloat16
    assert ((got["out"].double() - want["out"]).abs() <= tol).all()
    if case["lse"]:
        tol = dx + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * want["lse"].abs()
        assert ((got["lse"].double() - want["lse"]).abs() <= tol).all()
    else:
        assert got["lse"] is None


def _norm(case, seed, got):
    want = operators.exact({**case, "out": "both"}, seed)
    close = lambda a, b: ((a.double() - b).abs() <= (2.0 ** -8 + 2.0 ** -17) * b.abs()).all()
    assert (got["h"] is None) == (want["h"] is None) and (got["h"] is None or close(got["h"], want["h"]))
    assert (got["y"] is None) == (case["out"] == "fp8") and (got["y"] is None or close(got["y"], want["y"]))
    assert (got["y8"] is None) == (case["out"] == "bf16")
    if got["y8"] is not None:
        assert ((got["scale"].double() - want["scale"]).abs() <= 2.0 ** -17 * want["scale"]).all()
        D = case["dim"]
        wide = got["scale"].double().repeat_interleave(128 if case["group"] else D, dim=1)[:, :D]
        y = want["y"]
        tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * wide) * (1 + 2.0 ** -15) + 2.0 ** -16 * y.abs()
        assert ((got["y8"].double() * wide - y).abs() <= tol).all()


def _drawn(seed):
    return {**operators.draw(random.Random(seed)), "name": f"drawn_{seed}"}


@pytest.mark.gpu
@pytest.mark.parametrize("case", operators.listed() + [_drawn(s) for s in range(16)], ids=lambda c: c["name"])
def test_a_case_matches_its_definition(case, monkeypatch):
    build.build()
    monkeypatch.setattr(operators, "own", True)
    got = operators.run(operators.prepare(case, 5))
    assert api.dsa_get_device_error() == 0
    if case["op"] == "norm":
        _norm(case, 5, got)
    else:
        _attention(case, 5, got, monkeypatch)

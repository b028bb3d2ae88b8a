"""The measured cases of perf/more_operators.py, and some drawn from their ranges, against their float64 definitions.

Tolerances, as in the tests of each operator: with A = sum p |v| (exact probabilities), E the largest sm_scale * sum
|q||k| of a row and Q the largest sm_scale * max|q| * sum |k|, over n keys of D dims: scores are off by dx = D * 2^-24 E
(FP8 rows: 258 * 2^-24 E + 2^-17 Q + 2^-21 z, z = |x| / ln 2 + |log2 scale| at most), an output by 2^-8 |out| + (w + 2.1 dx +
n 2^-24 + 2^-18) A with w = 2^-8 (FP8: 2^-11, and n 2^-29 max|v| more), a log-sum-exp by dx + n 2^-24 + 2^-20 + 2^-23 |lse|.
Whole numbers are equal; copied rows too; a scale is off by 2^-23 of itself and a code by half a step, 2^-4 of the
quotient or 2^-10, and the quotient's 2^-22.
"""
import math
import random

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build
from perf import more_operators as ops


def test_cases_are_named_once_and_cover_every_operator():
    cases = ops.listed()
    assert len({c["name"] for c in cases}) == len(cases) and not ops.own
    assert {c["op"] for c in cases} == {"pages", "write", "decode", "prompt"}
    for seed in range(200):
        assert all(v > 0 for v in ops.work(ops.draw(random.Random(seed))).values())


def _bounds(q, k, v, limit, scale):
    """In place of an attention's (output, lse): (A, E)."""
    hide = torch.arange(k.shape[0], device=q.device)[None, :] >= limit[:, None]
    x = ((q @ k.T) * scale).masked_fill_(hide, float("-inf"))
    size = ((q.abs() @ k.abs().T) * scale).masked_fill_(hide, 0.0)
    return torch.softmax(x, dim=1) @ v.abs(), size.amax(dim=1)


def _query_bounds(q, k, v, limit, scale):
    """In place of an attention's (output, lse): (max|v|, Q + 2^-4 z), keys of a step taken for the whole request."""
    Q = scale * q.abs().amax(dim=1) * k.abs().sum(dim=1).amax()
    x = ((q @ k.T) * scale).abs().amax(dim=1)
    lg = torch.log2(v.abs().amax(dim=1).clamp(min=1e-30) / 448).abs().amax() + 9      # (a row's largest code: 2^-9 .. 448)
    return v.abs().amax().expand(q.shape[0], v.shape[1]), Q + 2.0 ** -4 * (x / math.log(2) + lg)


def _attention(case, seed, got, monkeypatch):
    whole, fp8 = {**case, "lse": True}, case.get("cache") == "fp8"
    want = ops.exact(whole, seed)
    monkeypatch.setattr(ops, "_attend64", _bounds)
    bound = ops.exact(whole, seed)
    A, E = bound["out"], bound["lse"]
    n = case["hi"] if case["op"] == "decode" else case["qhi"] + case["prefix"]
    dx, w, far = case["dim"] * 2.0 ** -24 * E, 2.0 ** -8, 0.0
    if fp8:
        monkeypatch.setattr(ops, "_attend64", _query_bounds)
        more = ops.exact(whole, seed)
        dx, w, far = 258 * 2.0 ** -24 * E + 2.0 ** -17 * more["lse"], 2.0 ** -11, n * 2.0 ** -29 * more["out"]
    tol = 2.0 ** -8 * want["out"].abs() + (w + 2.1 * dx[..., None] + n * 2.0 ** -24 + 2.0 ** -18) * A + far
    assert got["out"].dtype == torch.bfloat16
    assert ((got["out"].double() - want["out"]).abs() <= tol).all()
    if case["lse"]:
        tol = dx + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * want["lse"].abs()
        assert ((got["lse"].double() - want["lse"]).abs() <= tol).all()
    else:
        assert got["lse"] is None


def _write(case, seed, got, monkeypatch):
    monkeypatch.setattr(ops, "_e4m3", lambda quotient: quotient)
    want = ops.exact(case, seed)                 # copied values, or quotients before they are rounded to codes
    for name in ("k", "v"):
        if case["cache"] == "bf16":
            assert torch.equal(got[name].double(), want[name])
            continue
        s, x = want[name + "_scale"], want[name]
        assert ((got[name + "_scale"].double() - s).abs() <= 2.0 ** -23 * s).all()
        half = (2.0 ** -4 * x.abs()).clamp(min=2.0 ** -10)
        assert ((got[name].double() - x).abs() <= half + 2.0 ** -22 * x.abs()).all()


def _drawn(seed):
    return {**ops.draw(random.Random(seed)), "name": f"drawn_{seed}"}


@pytest.mark.gpu
@pytest.mark.parametrize("case", ops.listed() + [_drawn(s) for s in range(24)], ids=lambda c: c["name"])
def test_a_case_matches_its_definition(case, monkeypatch):
    build.build()
    monkeypatch.setattr(ops, "own", True)
    state = ops.prepare(case, 5)
    got = ops.run(state)
    assert api.dsa_get_device_error() == 0
    if case["op"] == "pages":
        want = ops.exact(case, 5)
        assert all(torch.equal(got[k], want[k]) for k in want)
        again = ops.run(state)
        assert all(torch.equal(again[k], want[k]) for k in want)
    elif case["op"] == "write":
        _write(case, 5, got, monkeypatch)
    else:
        _attention(case, 5, got, monkeypatch)

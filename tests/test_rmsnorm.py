"""The residual + root-mean-square norm with bf16 and FP8 output, against its formula in float64.

Tolerances, fixed beforehand: an output rounded to bf16 is off by at most half a step, 2^-8 of its
value; an E4M3 code by half a step, 2^-4 of its value, or half the subnormal step, 2^-10 of its scale.
The fp32 arithmetic before the rounding (a sum of squares over at most 32 terms a thread and ten
tree levels, a square root, a division, two products: under 64 roundings of 2^-24) adds 2^-18.
"""
import ctypes

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

ARITH = 2.0 ** -18
BF16, FP8 = 2.0 ** -8, 2.0 ** -4
FAKE = 0x7f0000000000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_refusals_on_the_host(L):
    ok = dict(rows=4, dim=256, x=FAKE, ld=256, residual=FAKE, weight=FAKE, eps=1e-6, group=128,
              residual_out=FAKE, y=FAKE, y8=FAKE, y_scale=FAKE)

    def call(**over):
        a = {**ok, **over}
        return L.dsa_rmsnorm(a["rows"], a["dim"], a["x"], a["ld"], a["residual"], a["weight"], a["eps"],
                             a["group"], a["residual_out"], a["y"], a["y8"], a["y_scale"], None)

    assert call(rows=0) == 0                                   # nothing to do
    for bad in (dict(rows=-1), dict(dim=0), dict(ld=248), dict(ld=260), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(weight=None),
                dict(residual=None), dict(residual_out=None), dict(y8=None), dict(y_scale=None),
                dict(y=None, y8=None, y_scale=None), dict(x=FAKE + 2), dict(weight=FAKE + 8),
                dict(residual=FAKE + 8), dict(residual_out=FAKE + 4), dict(y=FAKE + 8),
                dict(y8=FAKE + 4), dict(y_scale=FAKE + 2)):
        assert call(**bad) == 1, bad
    for bad in (dict(dim=252, ld=256), dict(dim=32776, ld=32776), dict(group=64), dict(group=1)):
        assert call(**bad) == 2, bad


def _formula(x, res, w, eps):
    h = x.double()
    if res is not None:
        h = h + res.double()
    return h, h / torch.sqrt((h * h).sum(1, keepdim=True) / x.shape[1] + eps) * w.double()


def _within(got, ref, rel, floor=0.0):
    bad = (got.double() - ref).abs() > rel * ref.abs() + floor
    assert not bad.any(), (got.double()[bad][:4], ref[bad][:4])


def _check_fp8(y8, scale, ref, group):
    T, D = ref.shape
    width = 128 if group else D
    for g in range(-(-D // width)):
        part = ref[:, g * width:(g + 1) * width]
        amax = part.abs().amax(1)
        want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        _within(scale[:, g], want, 2 * ARITH)
        codes = y8[:, g * width:(g + 1) * width].contiguous().view(torch.float8_e4m3fn).double()
        got = codes * scale[:, g:g + 1].double()
        bad = (got - part).abs() > torch.maximum(FP8 * part.abs(), 2.0 ** -10 * want[:, None]) * (1 + 8 * ARITH) + 4 * ARITH * part.abs()
        assert not bad.any()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,stride,group,residual,out", [
    (1, 8, 0, 128, False, "both"),            # one vector
    (3, 128, 0, 128, True, "fp8"),
    (5, 136, 0, 128, True, "both"),           # a tile of 8 columns at the end
    (9, 512, 576, 0, False, "bf16"),          # the latent's norm: a slice
    (17, 520, 528, 128, False, "both"),
    (33, 1608, 0, 128, True, "both"),
    (8, 4096, 0, 0, True, "fp8"),
    (2, 4104, 0, 128, True, "both"),
    (7, 8192, 8200, 0, False, "fp8"),
    (3, 16376, 0, 128, True, "both"),
    (2, 32768, 0, 0, True, "both"),
    (700, 5120, 0, 128, True, "fp8"),
])
def test_matches_formula(L, rows, dim, stride, group, residual, out):
    g = torch.Generator(device="cuda").manual_seed(rows * 1000 + dim)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    wide = (rnd(rows, stride or dim) * 3).to(torch.bfloat16)
    wide[:, dim:] = float("nan")              # outside the slice
    x = wide[:, :dim]
    if rows > 2:
        x[1] = 0                              # a row of zeros (with a residual: not)
        x[2, dim // 2:] = 0                   # tiles of zeros
    w = (1 + 0.3 * rnd(dim)).to(torch.bfloat16)
    res = rnd(rows, dim).to(torch.bfloat16) if residual else None
    eps = 1e-6
    h = torch.empty_like(res) if residual else None
    y = torch.empty((rows, dim), dtype=torch.bfloat16, device="cuda") if out != "fp8" else None
    y8 = torch.empty((rows, dim), dtype=torch.uint8, device="cuda") if out != "bf16" else None
    sc = torch.empty((rows, -(-dim // 128) if group else 1), device="cuda") if out != "bf16" else None
    api.dsa_rmsnorm(x, w, eps, residual=res, residual_out=h, y=y, y8=y8, y_scale=sc, group=group)
    h_ref, y_ref = _formula(x.cpu(), None if res is None else res.cpu(), w.cpu(), eps)
    if residual:
        _within(h.cpu(), h_ref, BF16 + ARITH)
    if y is not None:
        _within(y.cpu(), y_ref, BF16 + 2 * ARITH)
    if y8 is not None:
        _check_fp8(y8.cpu(), sc.cpu(), y_ref, group)


@pytest.mark.gpu
def test_in_place_on_another_stream_and_in_a_graph(L):
    g = torch.Generator(device="cuda").manual_seed(5)
    x0 = torch.randn(40, 1024, generator=g, device="cuda").to(torch.bfloat16)
    r0 = torch.randn(40, 1024, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(1024, generator=g, device="cuda").to(torch.bfloat16)
    want_h, want_y = torch.empty_like(x0), torch.empty_like(x0)
    api.dsa_rmsnorm(x0, w, 1e-5, residual=r0, residual_out=want_h, y=want_y)
    # the residual and x replaced in place
    x, r = x0.clone(), r0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.dsa_rmsnorm(x, w, 1e-5, residual=r, residual_out=r, y=x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(x, want_y) and torch.equal(r, want_h)
    # captured, replayed over new inputs
    xs, rs, ys = torch.zeros_like(x0), torch.zeros_like(r0), torch.empty_like(x0)
    hs = torch.empty_like(x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dsa_rmsnorm(xs, w, 1e-5, residual=rs, residual_out=hs, y=ys)
    xs.copy_(x0)
    rs.copy_(r0)
    graph.replay()
    assert torch.equal(ys, want_y) and torch.equal(hs, want_h)


@pytest.mark.gpu
def test_binding_checks_shapes(L):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y8 = torch.empty((4, 256), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_rmsnorm(x.cpu(), w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="CUDA"):
        api.dsa_rmsnorm(x, w, 1e-6, y=torch.empty((4, 256), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        api.dsa_rmsnorm(x.float(), w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(TypeError):
        api.dsa_rmsnorm(x[0], w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(TypeError):
        api.dsa_rmsnorm(x, w, 1e-6, y=torch.empty((4, 256), device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        api.dsa_rmsnorm(x, w, 1e-6, y=torch.empty((256, 4), dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="y_scale"):
        api.dsa_rmsnorm(x, w, 1e-6, y8=y8, y_scale=torch.empty((4, 1), device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        api.dsa_rmsnorm(x, w[:128], 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="columns"):
        api.dsa_rmsnorm(x.t(), w[:4], 1e-6, y=torch.empty((256, 4), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(api.DSAError):
        api.dsa_rmsnorm(x, w, 1e-6)
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    api.dsa_rmsnorm(empty, w, 1e-6, y=torch.empty_like(empty))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,group,residual", [
    (50, 1024, 0, False), (9, 1032, 128, False), (50, 1032, 0, True), (21, 1560, 128, False),
    (7, 2048, 128, True), (7, 2056, 0, False), (301, 3304, 128, False), (3, 4096, 128, False),
    (11, 6152, 0, True), (5, 12296, 128, False), (2, 32760, 128, False), (1, 64, 0, False),
])
def test_rows_that_share_a_block(L, rows, dim, group, residual):
    """Rows of one to 32 warps, several to a block where they are short, the last block not full."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    x, w, res = rnd(rows, dim), rnd(dim), rnd(rows, dim) if residual else None
    guard = torch.full((rows + 8, dim), 77.0, dtype=torch.bfloat16, device="cuda")
    y8 = torch.full((rows + 8, dim), 55, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows + 8, -(-dim // 128) if group else 1), 33.0, device="cuda")
    api.dsa_rmsnorm(x, w, 1e-5, residual=res, residual_out=None if res is None else torch.empty_like(res),
                    y=guard[:rows], y8=y8[:rows], y_scale=sc[:rows], group=group)
    assert (guard[rows:] == 77).all() and (y8[rows:] == 55).all() and (sc[rows:] == 33).all()
    _, ref = _formula(x.cpu(), None if res is None else res.cpu(), w.cpu(), 1e-5)
    _within(guard[:rows].cpu(), ref, BF16 + 2 * ARITH)
    _check_fp8(y8[:rows].cpu(), sc[:rows].cpu(), ref, group)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [256, 1032, 4104])
@pytest.mark.parametrize("group", [0, 128])
def test_tiny_and_undefined_rows(L, dim, group):
    g = torch.Generator(device="cuda").manual_seed(dim + group)
    x = torch.randn(8, dim, generator=g, device="cuda")
    x[1] *= 1e-33                             # the reciprocal of a tile's largest would overflow
    x[2, :128] *= 1e-36
    x[3], x[4, 5], x[6, dim - 1] = 0, float("nan"), float("nan")
    x = x.to(torch.bfloat16)
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")

    def run(eps):
        y, y8 = torch.empty_like(x), torch.empty((8, dim), dtype=torch.uint8, device="cuda")
        sc = torch.empty((8, -(-dim // 128) if group else 1), device="cuda")
        api.dsa_rmsnorm(x, w, eps, y=y, y8=y8, y_scale=sc, group=group)
        return y.cpu(), y8.cpu(), sc.cpu()

    y, y8, sc = run(1e-6)
    _, ref = _formula(x.cpu(), None, w.cpu(), 1e-6)
    good = torch.tensor([0, 1, 2, 3, 5, 7])
    # (Below 2^-126, bf16's steps are 2^-126 * 2^-7: a rounding there is off by 2^-134 at most.)
    _within(y[good], ref[good], BF16 + 2 * ARITH, floor=2.0 ** -134)
    _check_fp8(y8[good], sc[good], ref[good], group)
    # a NaN is its whole row's, in both outputs; so is 0 / 0 of a row of zeros without eps
    wide = lambda s: s.repeat_interleave(128 if group else dim, 1)[:, :dim]
    undefined = lambda y, y8, sc, r: y[r].isnan().all() and (
        y8.view(torch.float8_e4m3fn).float() * wide(sc))[r].isnan().all()
    assert undefined(y, y8, sc, 4) and undefined(y, y8, sc, 6)
    assert undefined(*run(0.0), 3)

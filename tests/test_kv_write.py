"""The cache write of layers with grouped heads: rows bit for bit in bf16; in FP8 the scale is amax / 448 in fp32
(off by 2^-23 of it at most) and a code times its scale is off by half a step of E4M3, 2^-4 of the value or 2^-10
of the scale (the smallest step's half), and by the quotient's rounding (2^-22 of the value, generously)."""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_refusals_on_the_host(L):
    ok = dict(tokens=5, heads=2, dim=128, k=FAKE, ld_k=256, v=FAKE, ld_v=256, slots=FAKE, pages=3, kc=FAKE, vc=FAKE)

    def call(fp8=False, **over):
        a = {**ok, **over}
        if not fp8:
            return L.dsa_kv_write(*a.values(), None)
        args = list(a.values())
        return L.dsa_kv_write_fp8(*args[:10], over.get("ks", FAKE), args[10], over.get("vs", FAKE), None)

    assert call(tokens=0) == 0 and call(True, tokens=0) == 0
    for fp8 in (False, True):
        for bad in (dict(tokens=-1), dict(heads=0), dict(pages=0), dict(ld_k=248), dict(ld_v=255), dict(ld_k=260),
                    dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(k=FAKE + 8),
                    dict(v=FAKE + 2), dict(slots=FAKE + 2), dict(kc=FAKE + 8), dict(vc=FAKE + 4)):
            assert call(fp8, **bad) == 1, bad
        for bad in (dict(dim=96), dict(dim=256), dict(heads=1025), dict(pages=1 << 25)):
            assert call(fp8, **bad) == 2, bad
    assert call(True, dim=64) == 2 and L.dsa_kv_write(5, 2, 64, FAKE, 255, FAKE, 256, FAKE, 3, FAKE, FAKE, None) == 1
    a = list(ok.values())
    assert L.dsa_kv_write_fp8(*a[:10], None, a[10], FAKE, None) == 1
    assert L.dsa_kv_write_fp8(*a[:10], FAKE, a[10], None, None) == 1


def _case(T, K, D, pages, wide, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, 2 * K * D + wide, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    x[T // 2, :] = 0                                     # a token of zeros
    k = x[:, wide:wide + K * D].unflatten(1, (K, D))
    v = x[:, wide + K * D:].unflatten(1, (K, D))
    slots = torch.randperm(pages * 64, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1
    return k, v, slots


SIZES = [(1, 1, 64, 1, 0), (1, 8, 128, 1, 8), (63, 3, 64, 2, 0), (65, 3, 128, 2, 24), (1000, 5, 128, 17, 0), (4001, 8, 128, 64, 1024),
         (257, 16, 64, 9, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,D,pages,wide", SIZES)
def test_bf16_rows_are_copied(L, T, K, D, pages, wide):
    k, v, slots = _case(T, K, D, pages, wide, T + K)
    caches = [torch.full((pages, K, 64, D), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    api.dsa_kv_write(k, v, slots, *caches)
    assert api.dsa_get_device_error() == 0
    for x, cache in zip((k, v), caches):
        want = torch.full((pages * 64, K, D), 77.0, dtype=torch.bfloat16, device="cuda")
        live = slots >= 0
        want[slots[live].long()] = x[live]
        assert torch.equal(cache, want.unflatten(0, (pages, 64)).transpose(1, 2).contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,D,pages,wide", [s for s in SIZES if s[2] == 128])
def test_fp8_rows(L, T, K, D, pages, wide):
    k, v, slots = _case(T, K, D, pages, wide, T + K)
    codes = [torch.full((pages, K, 64, D), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, K, 64), 77.0, device="cuda") for _ in range(2)]
    api.dsa_kv_write_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    assert api.dsa_get_device_error() == 0
    live = slots >= 0
    rows = slots[live].long()
    rest = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    rest[rows] = False
    for x, c, s in zip((k, v), codes, scales):
        c, s = c.transpose(1, 2).flatten(0, 1), s.transpose(1, 2).flatten(0, 1)
        assert (c[rest] == 77).all() and (s[rest] == 77).all()
        x, c, s = x[live].double(), c[rows].view(torch.float8_e4m3fn).double(), s[rows].double()
        top = x.abs().amax(dim=2)
        want = torch.where(top > 0, top / 448, 1.0)
        assert ((s - want).abs() <= 2.0 ** -23 * want).all()
        assert (c[top == 0] == 0).all()
        tol = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s[..., None]) + 2.0 ** -22 * x.abs()
        assert ((c * s[..., None] - x).abs() <= tol).all()


@pytest.mark.gpu
def test_codes_are_those_of_the_division(L):
    """Against amax / 448 and x / scale in fp32, rounded to E4M3: equal, but where the quotient lies next to a
    border between codes (at most one in ten thousand, off by one code)."""
    k, v, slots = _case(4096, 8, 128, 64, 0, 5)
    slots = torch.arange(4096, dtype=torch.int32, device="cuda")
    codes = [torch.empty((64, 8, 64, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty((64, 8, 64), device="cuda") for _ in range(2)]
    api.dsa_kv_write_fp8(k, v, slots, codes[0], scales[0], codes[1], scales[1])
    for x, c in zip((k, v), codes):
        x = x.float()
        top = x.abs().amax(dim=2, keepdim=True)
        # (By a tensor: a number as divisor becomes a product with its rounded reciprocal.)
        scale = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))
        want = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
        got = c.transpose(1, 2).flatten(0, 1)
        off = got != want
        assert off.float().mean() <= 1e-4
        assert ((got.int() - want.int()).abs()[off] <= 1).all()


@pytest.mark.gpu
def test_small_and_large_magnitudes(L):
    """Scales near both ends of the range, where a reciprocal or a remainder would be lost."""
    k = torch.ones(4, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[:, 0, ::2] = 0.3
    k[0] *= 2.0 ** -126
    k[1] *= 2.0 ** -110
    k[2] *= 2.0 ** 127
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    c, s = torch.empty((1, 1, 64, 128), dtype=torch.uint8, device="cuda"), torch.empty((1, 1, 64), device="cuda")
    api.dsa_kv_write_fp8(k, k, slots, c, s, c.clone(), s.clone())
    x = k[:, 0].float()
    scale = x.abs().amax(dim=1, keepdim=True)
    scale = scale / torch.full_like(scale, 448.0)
    assert torch.equal(s[0, 0, :4], scale[:, 0])
    assert torch.equal(c[0, 0, :4], (x / scale).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.gpu
def test_slots_outside_are_reported_and_skipped(L):
    k, v, slots = _case(40, 2, 128, 3, 0, 9)
    want = [torch.zeros((3, 2, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots[3] = slots[30] = slots[39] = -1
    api.dsa_kv_write(k, v, slots, *want)
    assert api.dsa_get_device_error() == 0
    slots[3], slots[30], slots[39] = 3 * 64, -2, 2 ** 31 - 1
    got = [torch.zeros_like(w) for w in want]
    api.dsa_kv_write(k, v, slots, *got)
    assert api.dsa_get_device_error() == 5
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_rows_past_two_to_the_31(L):
    """The last page of a cache of 2^32 values, from rows past 2^31 values of a projection."""
    pages, K, D = 65537 * 4, 2, 128
    cache = torch.empty((pages, K, 64, D), dtype=torch.bfloat16, device="cuda")
    cache[-1].zero_()
    rows = torch.empty((5, 1 << 30), dtype=torch.bfloat16, device="cuda")
    k = rows[:, :K * D].unflatten(1, (K, D))
    k.copy_(torch.randn(5, K, D, device="cuda"))
    slots = torch.arange(pages * 64 - 5, pages * 64, dtype=torch.int32, device="cuda")
    api.dsa_kv_write(k, k, slots, cache, torch.empty_like(cache))
    assert api.dsa_get_device_error() == 0
    assert torch.equal(cache[-1, :, 59:], k.transpose(0, 1)) and (cache[-1, :, :59] == 0).all()


@pytest.mark.gpu
def test_binding_checks(L):
    k, v, slots = _case(9, 2, 128, 1, 0, 1)
    cache = torch.zeros((1, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda k=k, v=v, slots=slots, a=cache, b=cache.clone(): api.dsa_kv_write(k, v, slots, a, b)
    call()
    with pytest.raises(ValueError, match="v:"):
        call(v=v[:, :1])
    with pytest.raises(ValueError, match="k: expected contiguous heads"):
        call(k=torch.zeros((9, 128, 2), dtype=torch.bfloat16, device="cuda").transpose(1, 2))
    with pytest.raises(TypeError, match="slots:"):
        call(slots=slots.long())
    with pytest.raises(ValueError, match="v_cache:"):
        call(b=cache[:, :1])
    with pytest.raises(TypeError, match="k_cache:"):
        call(a=cache.float())
    with pytest.raises(ValueError, match="k_scale:"):
        c8 = torch.zeros((1, 2, 64, 128), dtype=torch.uint8, device="cuda")
        api.dsa_kv_write_fp8(k, v, slots, c8, torch.ones((1, 2), device="cuda"), c8, torch.ones((1, 2, 64), device="cuda"))

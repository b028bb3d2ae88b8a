"""The operators beside the sparse layer run together, as a model's dense attention layer uses them: the
norm in front of the projections, the latent's norm, prompt attention over expanded keys and values, the
cache write, and decode in the absorbed form over the cache -- whose result for the tokens behind the
prompt has to be what the expanded form gives for the same tokens."""
import math

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

SM = 1.0 / math.sqrt(192.0)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,H", [([130, 64, 401], 1, 16), ([300, 77], 2, 32)])
def test_prompt_then_decode(lens, new, H):
    build.build()
    g = torch.Generator(device="cuda").manual_seed(new)
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    B, D, N = len(lens), 1024, sum(lens)
    w_norm, w_lat = (1 + 0.1 * rnd(D)).to(bf), (1 + 0.1 * rnd(512)).to(bf)
    w_down, w_q = (rnd(D, 576) / 32).to(bf), (rnd(D, H * 192) / 32).to(bf)
    w_uk, w_uv = (rnd(H, 512, 128) / math.sqrt(512)).to(bf), (rnd(H, 512, 128) / math.sqrt(512)).to(bf)

    # hidden states of all tokens (prompts and the `new` tokens behind each) -> norm -> projections
    x, res = rnd(N, D).to(bf), rnd(N, D).to(bf)
    h, y = torch.empty_like(x), torch.empty_like(x)
    y8, sc = torch.empty((N, D), dtype=torch.uint8, device="cuda"), torch.empty((N, D // 128), device="cuda")
    api.dsa_rmsnorm(x, w_norm, 1e-6, residual=res, residual_out=h, y=y, y8=y8, y_scale=sc)
    back = y8.view(torch.float8_e4m3fn).float().view(N, -1, 128) * sc[:, :, None]
    assert ((back.view(N, D) - y.float()).abs() <= (2.0 ** -4 + 2.0 ** -8) * y.float().abs() + 2.0 ** -9 * sc.amax()).all()
    down = y @ w_down
    latent = down.clone()
    api.dsa_rmsnorm(down[:, :512], w_lat, 1e-6, y=(normed := torch.empty((N, 512), dtype=bf, device="cuda")))
    latent[:, :512] = normed
    q = (y @ w_q).view(N, H, 192)

    # expanded form over all tokens
    kv = torch.cat([torch.einsum("nc,hcd->nhd", latent[:, :512], w_uk),
                    torch.einsum("nc,hcd->nhd", latent[:, :512], w_uv)], dim=2).contiguous()
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    out = torch.empty((N, H, 128), dtype=bf, device="cuda")
    api.dsa_mla_prefill(q, kv, latent[:, 512:], cu, cu, out, max(lens), SM)
    # ... and of the last tokens alone, as a chunk over the earlier ones
    last = torch.cat([torch.arange(int(cu[b + 1]) - new, int(cu[b + 1])) for b in range(B)]).cuda()
    cu_new = torch.arange(0, new * B + 1, new, dtype=torch.int32, device="cuda")
    chunk = torch.empty((new * B, H, 128), dtype=bf, device="cuda")
    api.dsa_mla_prefill(q[last].contiguous(), kv, latent[:, 512:], cu_new, cu, chunk, new, SM)
    assert (chunk.float() - out[last].float()).abs().max() <= 2.0 ** -6 * out.float().abs().max()

    # the cache: prompts' rows placed by the page table, the new tokens written by dsa_cache_write
    pages = [-(-n // 64) for n in lens]
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = ids[sum(pages[:b]):sum(pages[:b]) + n]
    cache = torch.zeros((sum(pages) * 64, 576), dtype=bf, device="cuda")
    for b, n in enumerate(lens):
        pos = torch.arange(n - new)
        rows = (table[b, pos // 64].long() * 64 + pos % 64).cuda()
        cache[rows] = latent[int(cu[b]):int(cu[b]) + n - new]
    table, seq = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    desc = api.make_desc(seq, table, new, H, 1, sum(pages))
    k_fp8 = torch.empty((cache.shape[0], 128), dtype=torch.uint8, device="cuda")
    k_scale = torch.empty(cache.shape[0], device="cuda")
    api.dsa_cache_write(desc, latent[last].contiguous(), rnd(new * B, 128).to(bf), cache, k_fp8, k_scale)

    # absorbed form: q_nope into the latent space, attention, out of it again
    qa = torch.cat([torch.einsum("nhd,hcd->nhc", q[last][..., :128].float(), w_uk.float()).to(bf),
                    q[last][..., 128:]], dim=2).contiguous()
    ws = torch.empty(api.dsa_mla_decode_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    for fp8 in (False, True):
        o = torch.empty((new * B, H, 512), dtype=bf, device="cuda")
        if fp8:
            rows = torch.empty((cache.shape[0], 656), dtype=torch.uint8, device="cuda")
            api.dsa_latent_to_fp8(cache, rows)
            api.dsa_mla_decode_fp8kv(desc, qa, rows, o, ws, SM)
        else:
            api.dsa_mla_decode(desc, qa, cache, o, ws, SM)
        got = torch.einsum("nhc,hcd->nhd", o.float(), w_uv.float())
        # The two forms round at different places (keys, values and the absorbed query to bf16: 2^-8 each of
        # terms whose sums cancel; FP8 rows: 2^-4); compared by their norms.
        err = (got - out[last].float()).norm() / out[last].float().norm()
        assert err <= (0.08 if fp8 else 0.02), err
    assert api.dsa_get_device_error() == 0

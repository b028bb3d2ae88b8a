"""The operators beside the sparse decode layer, as they are measured: dense latent attention over the
paged cache (absorbed form), prompt attention over expanded keys and values, and the residual +
root-mean-square norm with FP8 output.

Every case computes one call of one operator.  With ``own`` false, ``run`` takes the plain form (elementary
torch operations in fp32); with ``own`` true, the calls of the package's API.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, VDIM, ROPE, PAGE = 576, 512, 64, 64
NOPE = 128                      # non-rope dims of an expanded head's query and key
HEADV = 128                     # value dims of an expanded head
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


def listed():
    return [
        # One request of 4096 tokens with 16 heads (the smallest decode step: latency counts).
        dict(name="decode_tiny_4k", op="decode", batch=1, q=1, heads=16, lo=4096, hi=4096, cache="bf16", lse=True),
        # A large batch of short requests, where dense attention is what a sparse layer falls back to.
        dict(name="decode_short", op="decode", batch=128, q=1, heads=128, lo=512, hi=2048, cache="bf16", lse=False),
        # Verification of one drafted token: two queries a request over 32K tokens.
        dict(name="decode_mtp_32k", op="decode", batch=32, q=2, heads=128, lo=32769, hi=32769, cache="bf16", lse=False),
        # Long requests, one query each: the dense layers of a model whose other layers are sparse.
        dict(name="decode_long_128k", op="decode", batch=8, q=1, heads=128, lo=131072, hi=131072, cache="bf16", lse=True),
        # The same with ragged lengths over the FP8 latent cache (656-byte rows).
        dict(name="decode_varlen_fp8", op="decode", batch=8, q=1, heads=128, lo=65536, hi=131072, cache="fp8", lse=False),
        # One short prompt, 16 heads: latency.
        dict(name="prompt_short", op="prompt", batch=1, heads=16, qlo=77, qhi=77, prefix=0, causal=True, lse=True),
        # A batch of ragged prompts in one packed call.
        dict(name="prompt_ragged", op="prompt", batch=8, heads=128, qlo=200, qhi=2048, prefix=0, causal=True, lse=False),
        # One long prompt.
        dict(name="prompt_8k", op="prompt", batch=1, heads=128, qlo=8192, qhi=8192, prefix=0, causal=True, lse=False),
        # A prompt taken in chunks: 512 new tokens over an odd number of earlier ones.
        dict(name="prompt_chunk", op="prompt", batch=2, heads=128, qlo=512, qhi=512, prefix=16001, causal=True, lse=True),
        # The norm in front of a decode step's projections: few rows, 1 x 128 scale tiles.
        dict(name="norm_step", op="norm", rows=8, dim=5120, group=128, residual=True, out="fp8", stride=0),
        # The norm of a prompt's hidden states, one scale a token, the bf16 output as well.
        dict(name="norm_prompt", op="norm", rows=16384, dim=8192, group=0, residual=True, out="both", stride=0),
        # The latent's norm before it is cached: the first 512 of 576 columns, bf16 only.
        dict(name="norm_latent", op="norm", rows=32768, dim=512, group=0, residual=False, out="bf16", stride=576),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prompt", "norm"))
    if op == "decode":
        q = rng.choice((1, 1, 2, 3, 4))
        heads = rng.choice((16, 32, 48, 64, 80, 96, 112, 128))
        cache = rng.choice(("bf16", "bf16", "fp8"))
        hi = _log_int(rng, q, 131072)
        lo = max(q, int(hi * rng.uniform(0.3, 1.0)))
        tokens = 1000000 * 256 // max(256, q * heads)
        batch = _log_int(rng, 1, max(1, min(128, tokens // hi)))
        return dict(op=op, batch=batch, q=q, heads=heads, lo=lo, hi=hi, cache=cache,
                    lse=cache == "bf16" and rng.random() < 0.5)
    if op == "prompt":
        heads = rng.choice((8, 16, 24, 32, 64, 128))
        hi = _log_int(rng, 1, 6000)
        lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
        prefix = rng.choice((0, 0, _log_int(rng, 1, 16384)))
        pairs = heads * hi * (hi + prefix)
        batch = _log_int(rng, 1, max(1, min(16, int(4.0e9) // max(1, pairs))))
        return dict(op=op, batch=batch, heads=heads, qlo=lo, qhi=hi, prefix=prefix,
                    causal=rng.random() < 0.75, lse=rng.random() < 0.5)
    dim = 8 * _log_int(rng, 16, 2048)
    rows = _log_int(rng, 1, max(1, min(32768, (1 << 27) // dim)))
    residual = rng.random() < 0.6
    stride = 0 if residual or rng.random() < 0.5 else dim + 8 * rng.randint(1, 16)
    return dict(op=op, rows=rows, dim=dim, group=rng.choice((0, 128)), residual=residual,
                out=rng.choice(("fp8", "bf16", "both")), stride=stride)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    return g, host


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _fp8_rows(kv):
    """bf16 latent rows -> 656-byte FP8 rows: 512 E4M3 codes in four 128-value tiles, the tiles' fp32
    scales (amax / 448), the 64 rope values in bf16."""
    x = kv[:, :VDIM].float().view(-1, 4, 128)
    amax = x.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (x / scale[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, VDIM)
    return torch.cat([codes, scale.view(torch.uint8).view(-1, 16),
                      kv[:, VDIM:].contiguous().view(torch.uint8).view(-1, 2 * ROPE)], dim=1)


def prepare(case, seed):
    g, host = _gen(seed)
    return {"decode": _prepare_decode, "prompt": _prepare_prompt, "norm": _prepare_norm}[case["op"]](case, g, host)


def _prepare_decode(case, g, host):
    B, nq, H = case["batch"], case["q"], case["heads"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=host)
    pages = (lens + PAGE - 1) // PAGE
    num_pages, max_pages = int(pages.sum()), int(pages.max())
    phys = torch.randperm(num_pages, generator=host, dtype=torch.int64).to(torch.int32)
    col = torch.arange(max_pages)
    first = torch.cumsum(pages, 0) - pages
    at = (first[:, None] + col[None, :]).clamp(max=num_pages - 1)
    table = torch.where(col[None, :] < pages[:, None], phys[at], torch.tensor(-1, dtype=torch.int32))
    q = _randn(g, B * nq, H, LATENT)
    kv = _randn(g, num_pages * PAGE, LATENT)
    if case["cache"] == "fp8":
        kv = _fp8_rows(kv)
    s = dict(case=case, q=q, kv=kv, seqlens=lens.to(torch.int32).to(DEV), table=table.contiguous().to(DEV),
             num_pages=num_pages, max_len=int(lens.max()))
    if own:
        from deepseek_sparse_attention_lightning_gb300 import api
        s["desc"] = api.make_desc(s["seqlens"], s["table"], nq, H, 1, num_pages)
        s["ws"] = torch.empty(api.dsa_mla_decode_workspace_bytes(s["desc"]), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((B * nq, H, VDIM), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((B * nq, H), dtype=torch.float32, device=DEV) if case["lse"] else None
    return s


def _prompt_lens(case):
    """The prompts' lengths: the same for every seed, so that the packed outputs keep their shape."""
    host = torch.Generator()
    host.manual_seed(1000 * case["batch"] + case["qhi"])
    qlen = torch.randint(case["qlo"], case["qhi"] + 1, (case["batch"],), generator=host)
    return qlen, qlen + case["prefix"]


def _prepare_prompt(case, g, host):
    H = case["heads"]
    qlen, klen = _prompt_lens(case)
    zero = torch.zeros(1, dtype=torch.int64)
    cu_q = torch.cat([zero, torch.cumsum(qlen, 0)])
    cu_k = torch.cat([zero, torch.cumsum(klen, 0)])
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    latent = _randn(g, Tk, LATENT)     # the latent rows; the shared rope key is their last 64 columns
    s = dict(case=case, q=_randn(g, Tq, H, NOPE + ROPE), kv=_randn(g, Tk, H, NOPE + HEADV),
             k_rope=latent[:, VDIM:], cu_q=cu_q.to(torch.int32).to(DEV), cu_k=cu_k.to(torch.int32).to(DEV),
             max_q=int(qlen.max()), max_k=int(klen.max()))
    if own:
        s["out"] = torch.empty((Tq, H, HEADV), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((Tq, H), dtype=torch.float32, device=DEV) if case["lse"] else None
    return s


def _prepare_norm(case, g, host):
    T, D = case["rows"], case["dim"]
    x = _randn(g, T, case["stride"] or D)[:, :D]
    # Hidden states carry a few channels of large magnitude.
    loud = torch.ones(D, device=DEV)
    loud[torch.randperm(D, generator=host)[:max(1, D // 256)].to(DEV)] = 20.0
    x.mul_(loud.to(torch.bfloat16))
    s = dict(case=case, x=x, weight=(1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16),
             residual=_randn(g, T, D) * 2 if case["residual"] else None)
    if own:
        G = -(-D // 128) if case["group"] else 1
        s["h"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV) if case["residual"] else None
        s["y"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV) if case["out"] != "fp8" else None
        s["y8"] = torch.empty((T, D), dtype=torch.uint8, device=DEV) if case["out"] != "bf16" else None
        s["scale"] = torch.empty((T, G), dtype=torch.float32, device=DEV) if case["out"] != "bf16" else None
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"decode": _own_decode, "prompt": _own_prompt, "norm": _own_norm}[op](s)
    return {"decode": _plain_decode, "prompt": _plain_prompt, "norm": _plain_norm}[op](s)


def _own_decode(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    call = api.dsa_mla_decode if s["case"]["cache"] == "bf16" else api.dsa_mla_decode_fp8kv
    call(s["desc"], s["q"], s["kv"], s["out"], s["ws"], SM_SCALE, lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prompt(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    api.dsa_mla_prefill(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], s["out"], s["max_q"], SM_SCALE,
                        causal=s["case"]["causal"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_norm(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    api.dsa_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["h"], y=s["y"], y8=s["y8"],
                    y_scale=s["scale"], group=s["case"]["group"])
    return {"h": s["h"], "y": s["y"], "y8": None if s["y8"] is None else s["y8"].view(torch.float8_e4m3fn),
            "scale": s["scale"]}


def _plain_decode(s):
    case, q = s["case"], s["q"]
    B, nq, H = case["batch"], case["q"], case["heads"]
    pos = torch.arange(s["max_len"], device=DEV)
    page = s["table"].long().clamp_(min=0)[:, pos // PAGE]
    rows = s["kv"][page * PAGE + pos % PAGE]                                    # [B, S, row]
    if case["cache"] == "fp8":
        codes = rows[..., :VDIM].contiguous().view(torch.float8_e4m3fn).float()
        scale = rows[..., VDIM:VDIM + 16].contiguous().view(torch.float32)
        rope = rows[..., VDIM + 16:].contiguous().view(torch.bfloat16).float()
        value = (codes.view(B, -1, 4, 128) * scale[..., None]).view(B, -1, VDIM)
        key = torch.cat([value, rope], dim=2)
    else:
        key = rows.float()
        value = key[..., :VDIM]
    vis = s["seqlens"][:, None] - (nq - 1 - torch.arange(nq, device=DEV))[None, :]   # [B, nq]
    seen = (pos[None, None, :] < vis[:, :, None]).repeat_interleave(H, dim=1)        # [B, nq * H, S]
    x = torch.matmul(q.float().view(B, nq * H, LATENT), key.transpose(1, 2)).mul_(SM_SCALE)
    x = torch.where(seen, x, torch.tensor(-math.inf, device=DEV))
    m = x.amax(dim=2, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(dim=2, keepdim=True)
    out = (torch.matmul(p, value) / l).to(torch.bfloat16).view(B * nq, H, VDIM)
    return {"out": out, "lse": (m + torch.log(l)).view(B * nq, H) if case["lse"] else None}


def _plain_prompt(s):
    case = s["case"]
    qlen, klen = s["cu_q"].diff(), s["cu_k"].diff()
    qi = torch.arange(s["max_q"], device=DEV)
    ki = torch.arange(s["max_k"], device=DEV)
    qrow = (s["cu_q"][:-1, None] + qi[None, :]).clamp(max=s["q"].shape[0] - 1)
    krow = (s["cu_k"][:-1, None] + ki[None, :]).clamp(max=s["kv"].shape[0] - 1)
    q = s["q"][qrow].float().transpose(1, 2)                                    # [B, H, Q, 192]
    kv = s["kv"][krow].float().transpose(1, 2)                                  # [B, H, K, 256]
    rope = s["k_rope"][krow].float()[:, None]                                   # [B, 1, K, 64]
    x = torch.matmul(q[..., :NOPE], kv[..., :NOPE].transpose(2, 3))
    x.add_(torch.matmul(q[..., NOPE:], rope.transpose(2, 3))).mul_(SM_SCALE)
    seen = ki[None, None, :] < klen[:, None, None]
    if case["causal"]:
        seen = seen & (ki[None, None, :] <= (klen - qlen)[:, None, None] + qi[None, :, None])
    x.masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(dim=3, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(dim=3, keepdim=True)
    o = torch.matmul(x, kv[..., NOPE:]).div_(l).transpose(1, 2)                 # [B, Q, H, 128]
    valid = qi[None, :] < qlen[:, None]
    lse = (m + torch.log(l)).squeeze(3).transpose(1, 2)[valid] if case["lse"] else None
    return {"out": o[valid].to(torch.bfloat16), "lse": lse}


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    T, D = x.shape
    h = x if s["residual"] is None else x + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    got = {"h": None if s["residual"] is None else h.to(torch.bfloat16), "y": None, "y8": None, "scale": None}
    if case["out"] != "fp8":
        got["y"] = y.to(torch.bfloat16)
    if case["out"] != "bf16":
        width = 128 if case["group"] else D
        G = -(-D // width)
        tiles = torch.nn.functional.pad(y, (0, G * width - D)).view(T, G, width)
        amax = tiles.abs().amax(dim=2, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        got["y8"] = (tiles / scale).view(T, G * width)[:, :D].to(torch.float8_e4m3fn)
        got["scale"] = scale.view(T, G)
    return got


def work(case):
    if case["op"] == "decode":
        B, nq, H = case["batch"], case["q"], case["heads"]
        keys = B * (case["lo"] + case["hi"]) / 2
        row = 656 if case["cache"] == "fp8" else 2 * LATENT
        pairs = B * sum((case["lo"] + case["hi"]) / 2 - (nq - 1 - i) for i in range(nq)) * H
        return {"bytes": keys * row + B * nq * H * 2 * (LATENT + VDIM) + (B * nq * H * 4 if case["lse"] else 0),
                "flops": pairs * 2 * (LATENT + VDIM)}
    if case["op"] == "prompt":
        H = case["heads"]
        qlen, klen = (n.double() for n in _prompt_lens(case))
        pairs = float((qlen * (klen - qlen) + qlen * (qlen + 1) / 2 if case["causal"] else qlen * klen).sum())
        nq, nk = float(qlen.sum()), float(klen.sum())
        return {"bytes": nq * H * (2 * (NOPE + ROPE + HEADV) + (4 if case["lse"] else 0))
                + nk * 2 * (H * (NOPE + HEADV) + ROPE),
                "flops": pairs * H * 2 * (NOPE + ROPE + HEADV)}
    T, D = case["rows"], case["dim"]
    moved = 2 + (4 if case["residual"] else 0) + (0 if case["out"] == "fp8" else 2) + (0 if case["out"] == "bf16" else 1)
    scales = 0 if case["out"] == "bf16" else T * 4 * (-(-D // 128) if case["group"] else 1)
    return {"bytes": T * D * moved + 2 * D + scales, "flops": T * D * 6}


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "prompt": _exact_prompt, "norm": _exact_norm}[case["op"]](s)


def _attend64(q, k, v, limit):
    """Softmax attention of one head group in fp64: q [n, d], k [s, d], v [s, e]; row i sees keys < limit[i]."""
    x = (q @ k.T) * SM_SCALE
    x[torch.arange(k.shape[0], device=DEV)[None, :] >= limit[:, None]] = -math.inf
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse[:, None]) @ v, lse


def _exact_decode(s):
    case = s["case"]
    nq, H = case["q"], case["heads"]
    outs, lses = [], []
    for r, n in enumerate(s["seqlens"].tolist()):
        at = s["table"][r, :-(-n // PAGE)].long()
        rows = s["kv"].view(s["num_pages"], PAGE, -1)[at].flatten(0, 1)[:n]
        if case["cache"] == "fp8":
            sc = rows[:, 512:528].contiguous().view(torch.float32).double()
            c = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double()
            v = c * sc.repeat_interleave(128, dim=1)
            k = torch.cat([v, rows[:, 528:].contiguous().view(torch.bfloat16).double()], dim=1)
        else:
            k = rows.double()
            v = k[:, :VDIM]
        limit = torch.arange(n - nq + 1, n + 1, device=DEV).repeat_interleave(H)
        o, e = _attend64(s["q"][r * nq:(r + 1) * nq].double().flatten(0, 1), k, v, limit)
        outs.append(o.view(nq, H, VDIM))
        lses.append(e.view(nq, H))
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}


def _exact_prompt(s):
    case = s["case"]
    out = torch.empty((s["q"].shape[0], case["heads"], HEADV), dtype=torch.float64, device=DEV)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEV)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        q0, q1, k0, k1 = cq[b], cq[b + 1], ck[b], ck[b + 1]
        n, m = q1 - q0, k1 - k0
        limit = (torch.arange(n, device=DEV) + (m - n + 1)) if case["causal"] else torch.full((n,), m, device=DEV)
        rope = s["k_rope"][k0:k1].double()
        for h in range(case["heads"]):
            kv = s["kv"][k0:k1, h].double()
            o, e = _attend64(s["q"][q0:q1, h].double(), torch.cat([kv[:, :NOPE], rope], dim=1), kv[:, NOPE:], limit)
            out[q0:q1, h] = o
            lse[q0:q1, h] = e
    return {"out": out, "lse": lse if case["lse"] else None}


def _e4m3(v):
    """fp64 values rounded to the nearest E4M3 value (ties to even), at most 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(s):
    case = s["case"]
    T, D = s["x"].shape
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / D + EPS) * s["weight"].double()
    got = {"h": h if s["residual"] is not None else None, "y": y if case["out"] != "fp8" else None,
           "y8": None, "scale": None}
    if case["out"] != "bf16":
        parts = torch.split(y, 128 if case["group"] else D, dim=1)
        scale = torch.stack([p.abs().amax(dim=1) for p in parts], dim=1) / 448.0
        scale[scale == 0] = 1.0
        got["scale"] = scale
        got["y8"] = torch.cat([_e4m3(p / scale[:, i:i + 1]) for i, p in enumerate(parts)], dim=1)
    return got

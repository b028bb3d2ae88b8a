"""The operators of layers with grouped heads, as they are measured: the page table and slot map of a step,
the write of its keys and values to the paged cache, attention of new tokens over that cache, and attention
over packed prompts.

Every case computes one call of one operator.  With ``own`` false, ``run`` takes the plain form (elementary
torch operations in fp32); with ``own`` true, the calls of the package's API.

H query heads share K key / value heads (H / K each); D is the dims of a head.  A cache is
[num_pages, K, 64, D]: a page of a head is contiguous.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64


def listed():
    return [
        # A decode step's bookkeeping: one new token for each of 128 requests.
        dict(name="pages_step", op="pages", batch=128, lo=1, hi=131072, add_lo=1, add_hi=1, spare=64),
        # A wave of ragged prompts enters empty rows: tables and slots of half a million tokens.
        dict(name="pages_prompts", op="pages", batch=256, lo=0, hi=0, add_lo=1, add_hi=4096, spare=1000),
        # The step's keys and values, one token a request, copied to bf16 rows.
        dict(name="write_step", op="write", tokens=128, kv_heads=8, dim=128, cache="bf16", fused=True),
        # A prompt chunk's keys and values, quantised to FP8 rows; an odd number of tokens.
        dict(name="write_prompt_fp8", op="write", tokens=32767, kv_heads=8, dim=128, cache="fp8", fused=True),
        # One request of 4000 tokens (the smallest decode step: latency counts).
        dict(name="decode_one_4k", op="decode", batch=1, q=1, heads=32, kv_heads=8, dim=128, lo=4000, hi=4000,
             cache="bf16", lse=True),
        # A batch of ragged requests with a drafted token each, 64-dim heads.
        dict(name="decode_ragged_mtp", op="decode", batch=64, q=2, heads=32, kv_heads=8, dim=64, lo=512, hi=16384,
             cache="bf16", lse=False),
        # Long requests, one query each.
        dict(name="decode_long_128k", op="decode", batch=8, q=1, heads=64, kv_heads=8, dim=128, lo=131072,
             hi=131072, cache="bf16", lse=True),
        # Ragged long requests over FP8 rows, and a group size that is no power of two.
        dict(name="decode_varlen_fp8", op="decode", batch=32, q=1, heads=40, kv_heads=8, dim=128, lo=16384,
             hi=65536, cache="fp8", lse=False),
        # One short prompt: latency.
        dict(name="prompt_short", op="prompt", batch=1, heads=32, kv_heads=8, dim=128, qlo=77, qhi=77, prefix=0,
             causal=True, lse=True),
        # A batch of ragged prompts in one packed call, 64-dim heads.
        dict(name="prompt_ragged", op="prompt", batch=16, heads=32, kv_heads=8, dim=64, qlo=200, qhi=2048, prefix=0,
             causal=True, lse=False),
        # One long prompt.
        dict(name="prompt_8k", op="prompt", batch=1, heads=64, kv_heads=8, dim=128, qlo=8192, qhi=8192, prefix=0,
             causal=True, lse=False),
        # Prompts taken in chunks: 512 new tokens over an odd number of earlier ones, five heads a group.
        dict(name="prompt_chunk", op="prompt", batch=4, heads=40, kv_heads=8, dim=128, qlo=512, qhi=512,
             prefix=16001, causal=True, lse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("pages", "write", "decode", "decode", "prompt", "prompt"))
    if op == "pages":
        batch = _log_int(rng, 1, 2048)
        add_hi = _log_int(rng, 1, max(1, min(4096, (1 << 19) // batch)))
        hi = rng.choice((0, _log_int(rng, 1, 131072)))
        return dict(op=op, batch=batch, lo=hi // 4, hi=hi, add_lo=rng.choice((0, (add_hi + 1) // 2)), add_hi=add_hi,
                    spare=rng.randint(0, 2000))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16) if g * kv_heads <= 128])
    if op == "write":
        cache = rng.choice(("bf16", "fp8"))
        dim = 128 if cache == "fp8" else dim
        tokens = _log_int(rng, 1, min(131072, (1 << 24) // (kv_heads * dim)))
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, cache=cache, fused=rng.random() < 0.7)
    heads = group * kv_heads
    if op == "decode":
        cache = rng.choice(("bf16", "bf16", "fp8"))
        dim = 128 if cache == "fp8" else dim
        q = rng.choice((1, 1, 1, 2, 3, 4))
        hi = _log_int(rng, q, 131072)
        lo = max(q, int(hi * rng.uniform(0.2, 1.0)))
        tokens = 8000000 // max(kv_heads, q * heads // 8)
        batch = _log_int(rng, 1, max(1, min(256, tokens // hi)))
        return dict(op=op, batch=batch, q=q, heads=heads, kv_heads=kv_heads, dim=dim, lo=lo, hi=hi, cache=cache,
                    lse=rng.random() < 0.5)
    hi = _log_int(rng, 1, 6000)
    prefix = rng.choice((0, 0, _log_int(rng, 1, 16384)))
    most = int(2.0e9)                                       # pairs of a query and a key, over the heads
    while heads * hi * (hi + prefix) > most:
        hi, prefix = hi * 3 // 4, prefix * 3 // 4
    lo = max(1, int(hi * rng.uniform(0.2, 1.0)))
    batch = _log_int(rng, 1, max(1, min(32, most // (heads * hi * (hi + prefix)))))
    return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, qlo=lo, qhi=hi, prefix=prefix,
                causal=rng.random() < 0.8, lse=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    return g, host


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _fixed_lens(case, lo, hi, salt):
    """Lengths that are the same for every seed, so that packed outputs keep their shape."""
    host = torch.Generator()
    host.manual_seed(1000 * case["batch"] + hi + salt)
    return torch.randint(lo, hi + 1, (case["batch"],), generator=host)


def _added(case):
    """New tokens of each request: the first has some."""
    add = _fixed_lens(case, case["add_lo"], case["add_hi"], 7)
    add[0] = max(1, int(add[0]))
    return add


def prepare(case, seed):
    g, host = _gen(seed)
    return {"pages": _prepare_pages, "write": _prepare_write, "decode": _prepare_decode,
            "prompt": _prepare_prompt}[case["op"]](case, g, host)


def _prepare_pages(case, g, host):
    B = case["batch"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=host)
    add = _added(case)
    held = (lens + PAGE - 1) // PAGE
    after = (lens + add + PAGE - 1) // PAGE
    used, total = int(held.sum()), int(after.sum())
    num_pages = total + case["spare"]
    phys = torch.randperm(num_pages, generator=host, dtype=torch.int64).to(torch.int32)
    max_pages = max(1, (case["hi"] + case["add_hi"] + PAGE - 1) // PAGE)
    col = torch.arange(max_pages)
    first = torch.cumsum(held, 0) - held
    at = (first[:, None] + col[None, :]).clamp(max=num_pages - 1)
    table = torch.where(col[None, :] < held[:, None], phys[at], torch.tensor(-1, dtype=torch.int32))
    free = torch.full((num_pages,), -1, dtype=torch.int32)
    free[:num_pages - used] = phys[used:]
    tokens = int(add.sum())
    i32 = lambda t: t.to(torch.int32).to(DEV)
    s = dict(case=case, seqlens=i32(lens), add=i32(add), table=table.contiguous().to(DEV), free=free.to(DEV),
             free_count=i32(torch.tensor([num_pages - used])), tokens=tokens, num_pages=num_pages)
    if own:
        s["cu"] = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(max(1, tokens), dtype=torch.int32, device=DEV)
        s["seqlens_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["free_count_out"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return s


def _prepare_write(case, g, host):
    T, K, D = case["tokens"], case["kv_heads"], case["dim"]
    num_pages = -(-T // PAGE) + 3
    # New tokens of a step lie anywhere, a prompt's page by page.
    if T <= 1024:
        slots = torch.randperm(num_pages * PAGE, generator=host)[:T]
    else:
        slots = (torch.randperm(num_pages, generator=host)[:, None] * PAGE + torch.arange(PAGE)[None, :]).flatten()[:T]
    slots[1:][torch.rand(T - 1, generator=host) < 0.01] = -1        # padding of the batch
    if case["fused"]:
        rows = _randn(g, T, 2 * K * D + 4 * D)              # a projection whose first columns are queries
        k, v = rows[:, 4 * D:4 * D + K * D], rows[:, 4 * D + K * D:]
    else:
        k, v = _randn(g, T, K * D), _randn(g, T, K * D)
    s = dict(case=case, k=k.unflatten(1, (K, D)), v=v.unflatten(1, (K, D)), slots=slots.to(torch.int32).to(DEV),
             num_pages=num_pages)
    shape = (num_pages, K, PAGE, D)
    if case["cache"] == "bf16":
        s["caches"] = [torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    else:
        s["caches"] = [torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2)]
        s["scales"] = [torch.ones(shape[:3], device=DEV) for _ in range(2)]
    return s


def _prepare_decode(case, g, host):
    B, nq, H, K, D = case["batch"], case["q"], case["heads"], case["kv_heads"], case["dim"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=host)
    pages = (lens + PAGE - 1) // PAGE
    num_pages, max_pages = int(pages.sum()), int(pages.max())
    phys = torch.randperm(num_pages, generator=host, dtype=torch.int64).to(torch.int32)
    col = torch.arange(max_pages)
    first = torch.cumsum(pages, 0) - pages
    at = (first[:, None] + col[None, :]).clamp(max=num_pages - 1)
    table = torch.where(col[None, :] < pages[:, None], phys[at], torch.tensor(-1, dtype=torch.int32))
    q = _randn(g, B * nq, H, D)
    s = dict(case=case, q=q, seqlens=lens.to(torch.int32).to(DEV), table=table.contiguous().to(DEV),
             num_pages=num_pages, max_len=int(lens.max()), lens=lens.tolist())
    shape = (num_pages, K, PAGE, D)
    if case["cache"] == "bf16":
        s["caches"] = [_randn(g, *shape), _randn(g, *shape)]
    else:
        s["caches"], s["scales"] = [], []
        for _ in range(2):
            x = _randn(g, *shape)
            scale = x.abs().amax(dim=3).float() / 448.0
            s["scales"].append(scale)
            s["caches"].append(torch.cat([(p.float() / c[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                                          for p, c in zip(x.split(4096), scale.split(4096))]))
    if own:
        from deepseek_sparse_attention_lightning_gb300 import api
        s["desc"] = api.make_desc(s["seqlens"], s["table"], nq, H, 1, num_pages)
        s["ws"] = torch.empty(api.dsa_gqa_decode_workspace_bytes(s["desc"], K, D), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((B * nq, H, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((B * nq, H), dtype=torch.float32, device=DEV) if case["lse"] else None
    return s


def _prompt_lens(case):
    qlen = _fixed_lens(case, case["qlo"], case["qhi"], 0)
    return qlen, qlen + case["prefix"]


def _prepare_prompt(case, g, host):
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    qlen, klen = _prompt_lens(case)
    zero = torch.zeros(1, dtype=torch.int64)
    cu_q = torch.cat([zero, torch.cumsum(qlen, 0)])
    cu_k = torch.cat([zero, torch.cumsum(klen, 0)])
    Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
    if case["prefix"] == 0:                     # one projection holds queries, keys and values
        rows = _randn(g, Tq, (H + 2 * K) * D)
        q, k, v = rows.split([H * D, K * D, K * D], dim=1)
    else:
        q, k, v = _randn(g, Tq, H * D), _randn(g, Tk, K * D), _randn(g, Tk, K * D)
    s = dict(case=case, q=q.unflatten(1, (H, D)), k=k.unflatten(1, (K, D)), v=v.unflatten(1, (K, D)),
             cu_q=cu_q.to(torch.int32).to(DEV), cu_k=cu_k.to(torch.int32).to(DEV), max_q=int(qlen.max()),
             qlens=qlen.tolist(), klens=klen.tolist())
    if own:
        s["out"] = torch.empty((Tq, H, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((Tq, H), dtype=torch.float32, device=DEV) if case["lse"] else None
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"pages": _own_pages, "write": _own_write, "decode": _own_decode, "prompt": _own_prompt}[op](s)
    return {"pages": _plain_pages, "write": _plain_write, "decode": _plain_decode, "prompt": _plain_prompt}[op](s)


def _fp8_values(c):
    return c.view(torch.float8_e4m3fn)


def _written(s):
    if s["case"]["cache"] == "bf16":
        return {"k": s["caches"][0], "v": s["caches"][1]}
    return {"k": _fp8_values(s["caches"][0]), "v": _fp8_values(s["caches"][1]), "k_scale": s["scales"][0],
            "v_scale": s["scales"][1]}


def _own_pages(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    # (Lengths and count go to buffers of their own, so that a pass can be made again.)
    api.dsa_pages_update(s["add"], s["seqlens"], s["table"], s["free"], s["free_count"], s["cu"],
                         s["slots"], seqlens_out=s["seqlens_out"], free_count_out=s["free_count_out"])
    return {"table": s["table"], "seqlens": s["seqlens_out"], "free_count": s["free_count_out"], "cu": s["cu"],
            "slots": s["slots"][:s["tokens"]]}


def _own_write(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    if s["case"]["cache"] == "bf16":
        api.dsa_kv_write(s["k"], s["v"], s["slots"], *s["caches"])
    else:
        api.dsa_kv_write_fp8(s["k"], s["v"], s["slots"], s["caches"][0], s["scales"][0], s["caches"][1],
                             s["scales"][1])
    return _written(s)


def _own_decode(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    scale = s["case"]["dim"] ** -0.5
    if s["case"]["cache"] == "bf16":
        api.dsa_gqa_decode(s["desc"], s["q"], *s["caches"], s["out"], s["ws"], scale, lse=s["lse"])
    else:
        api.dsa_gqa_decode_fp8kv(s["desc"], s["q"], s["caches"][0], s["scales"][0], s["caches"][1], s["scales"][1],
                                 s["out"], s["ws"], scale, lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prompt(s):
    from deepseek_sparse_attention_lightning_gb300 import api
    api.dsa_gqa_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["max_q"],
                        s["case"]["dim"] ** -0.5, causal=s["case"]["causal"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_pages(s):
    lens, add, table = s["seqlens"].long(), s["add"].long(), s["table"]
    held = (lens + PAGE - 1) // PAGE
    need = (lens + add + PAGE - 1) // PAGE - held
    before = torch.cumsum(need, 0) - need
    # New entries of the table, from the top of the free stack.
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    at = s["free_count"].long() - 1 - (before[:, None] + col - held[:, None])
    new = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(new, s["free"][at.clamp(0, s["num_pages"] - 1)], table)
    # The tokens' cache rows.
    ends = torch.cumsum(add, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends])
    r = torch.repeat_interleave(add, output_size=s["tokens"])
    pos = lens[r] + torch.arange(s["tokens"], device=DEV) - cu[r]
    slots = table[r, pos // PAGE] * PAGE + (pos % PAGE).to(torch.int32)
    return {"table": table, "seqlens": (lens + add).to(torch.int32),
            "free_count": (s["free_count"] - need.sum()).to(torch.int32), "cu": cu.to(torch.int32), "slots": slots}


def _plain_write(s):
    # Tokens without a slot write the first token's row again (it has one).
    live = s["slots"] >= 0
    keep = torch.where(live, torch.arange(live.shape[0], device=DEV), 0)
    slots = s["slots"][keep].long()
    page, row = slots // PAGE, slots % PAGE
    for i, x in enumerate((s["k"], s["v"])):
        x = x[keep]
        if s["case"]["cache"] == "bf16":
            s["caches"][i][page, :, row] = x
            continue
        x = x.float()
        amax = x.abs().amax(dim=2)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        s["caches"][i][page, :, row] = (x / scale[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scales"][i][page, :, row] = scale
    return _written(s)


def _plain_decode(s):
    case = s["case"]
    B, nq, H, K, D = case["batch"], case["q"], case["heads"], case["kv_heads"], case["dim"]
    G = H // K
    outs, lses = [], []
    step = max(1, 262144 // (s["max_len"] * K // 8 + 1))        # requests at a time
    for r0 in range(0, B, step):
        lens, b = s["seqlens"][r0:r0 + step], min(step, B - r0)
        n = -(-max(s["lens"][r0:r0 + step]) // PAGE)
        page = s["table"][r0:r0 + step, :n].long().clamp(min=0)
        k, v = (c[page] for c in s["caches"])                                   # [b, n, K, 64, D]
        if case["cache"] == "fp8":
            k, v = (_fp8_values(x).float() * c[page][..., None] for x, c in zip((k, v), s["scales"]))
        k, v = (x.float().transpose(1, 2).reshape(b, K, n * PAGE, D) for x in (k, v))
        q = s["q"][r0 * nq:(r0 + b) * nq].float().view(b, nq, K, G, D).permute(0, 2, 1, 3, 4).reshape(b, K, nq * G, D)
        x = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5)
        vis = (lens[:, None] - (nq - 1 - torch.arange(nq, device=DEV))[None, :]).repeat_interleave(G, dim=1)
        hide = torch.arange(n * PAGE, device=DEV)[None, None, :] >= vis[:, :, None]
        x.masked_fill_(hide[:, None], -math.inf)
        m = x.amax(dim=3, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(dim=3, keepdim=True)
        back = lambda t: t.view(b, K, nq, G, -1).permute(0, 2, 1, 3, 4).reshape(b * nq, H, -1)
        outs.append(back((torch.matmul(p, v) / l).to(torch.bfloat16)))
        lses.append(back(m + torch.log(l)).squeeze(2))
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}


def _plain_prompt(s):
    case = s["case"]
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // K
    outs, lses = [], []
    a = b = 0
    for n, m in zip(s["qlens"], s["klens"]):
        q = s["q"][a:a + n].float().view(n, K, G, D).permute(1, 2, 0, 3).reshape(K, G * n, D)
        k, v = (x[b:b + m].float().transpose(0, 1) for x in (s["k"], s["v"]))   # [K, m, D]
        x = torch.matmul(q, k.transpose(1, 2)).mul_(D ** -0.5).view(K, G, n, m)
        if case["causal"]:
            hide = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
            x.masked_fill_(hide, -math.inf)
        top = x.amax(dim=3, keepdim=True)
        x.sub_(top).exp_()
        l = x.sum(dim=3, keepdim=True)
        o = torch.matmul(x.view(K, G * n, m), v).view(K, G, n, D).div_(l)
        outs.append(o.permute(2, 0, 1, 3).reshape(n, H, D).to(torch.bfloat16))
        lses.append((top + torch.log(l)).squeeze(3).permute(2, 0, 1).reshape(n, H))
        a, b = a + n, b + m
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}


def work(case):
    if case["op"] == "pages":
        B = case["batch"]
        add = _added(case).double()
        tokens = float(add.sum())
        pages = tokens / PAGE + B * 0.5 * (1.0 if case["hi"] == 0 else 0.0)      # new ones, about
        return {"bytes": 4.0 * (tokens + 2 * pages + 4 * B + 3), "flops": 4.0 * tokens}
    if case["op"] == "write":
        values = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        if case["cache"] == "bf16":
            return {"bytes": 4 * values + 4 * case["tokens"], "flops": values}
        return {"bytes": 3 * values + 8 * case["tokens"] * case["kv_heads"] + 4 * case["tokens"], "flops": 3 * values}
    D, H, K = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "decode":
        B, nq = case["batch"], case["q"]
        mean = (case["lo"] + case["hi"]) / 2
        row = K * (2 * D + 8 if case["cache"] == "fp8" else 4 * D)
        pairs = B * sum(mean - (nq - 1 - i) for i in range(nq)) * H
        return {"bytes": B * mean * row + B * nq * H * (4 * D + (4 if case["lse"] else 0)), "flops": pairs * 4 * D}
    qlen, klen = (n.double() for n in _prompt_lens(case))
    pairs = float((qlen * (klen - qlen) + qlen * (qlen + 1) / 2 if case["causal"] else qlen * klen).sum())
    nq, nk = float(qlen.sum()), float(klen.sum())
    return {"bytes": nq * H * (4 * D + (4 if case["lse"] else 0)) + nk * K * 4 * D, "flops": pairs * H * 4 * D}


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "write": _exact_write, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](s)


def _exact_pages(s):
    """By a walk over the requests, on the host."""
    lens, add, table = s["seqlens"].tolist(), s["add"].tolist(), s["table"].tolist()
    free, count = s["free"].tolist(), int(s["free_count"])
    cu, slots = [0], []
    for r, n in enumerate(add):
        have = -(-lens[r] // PAGE)
        while have * PAGE < lens[r] + n:
            count -= 1
            table[r][have] = free[count]
            have += 1
        slots += [table[r][p // PAGE] * PAGE + p % PAGE for p in range(lens[r], lens[r] + n)]
        lens[r] += n
        cu.append(cu[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    return {"table": i32(table), "seqlens": i32(lens), "free_count": i32([count]), "cu": i32(cu), "slots": i32(slots)}


def _e4m3(v):
    """fp64 values rounded to the nearest E4M3 value (ties to even), at most 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_write(s):
    case = s["case"]
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    rows = s["slots"][live].long()
    got = {}
    for i, name in enumerate(("k", "v")):
        x = s["k" if i == 0 else "v"][live].double()                            # [n, K, D]
        cache = torch.zeros(s["num_pages"] * PAGE, case["kv_heads"], case["dim"], dtype=torch.float64, device=DEV)
        paged = lambda t: t.unflatten(0, (s["num_pages"], PAGE)).transpose(1, 2)
        if case["cache"] == "fp8":
            top = x.abs().max(dim=2).values
            scale = torch.where(top > 0, top / 448.0, 1.0)
            x = _e4m3(x / scale[..., None])
            scales = torch.ones(cache.shape[:2], dtype=torch.float64, device=DEV)
            scales[rows] = scale
            got[name + "_scale"] = paged(scales)
        cache[rows] = x
        got[name] = paged(cache)
    return {name: got[name] for name in ("k", "v", "k_scale", "v_scale") if name in got}


def _attend64(q, k, v, limit, scale):
    """Softmax attention in fp64: q [n, d], k, v [s, d]; row i sees keys < limit[i]."""
    x = (q @ k.T) * scale
    x[torch.arange(k.shape[0], device=DEV)[None, :] >= limit[:, None]] = -math.inf
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse[:, None]) @ v, lse


def _exact_decode(s):
    case = s["case"]
    nq, H, K, D = case["q"], case["heads"], case["kv_heads"], case["dim"]
    G = H // K
    out = torch.empty((case["batch"], nq, K, G, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((case["batch"], nq, K, G), dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"]):
        at = s["table"][r, :-(-n // PAGE)].long()
        limit = torch.arange(n - nq + 1, n + 1, device=DEV).repeat_interleave(G)
        for h in range(K):
            kv = []
            for i in range(2):
                x = s["caches"][i][at, h].flatten(0, 1)[:n]
                if case["cache"] == "fp8":
                    x = _fp8_values(x).double() * s["scales"][i][at, h].flatten()[:n, None].double()
                kv.append(x.double())
            q = s["q"][r * nq:(r + 1) * nq, h * G:(h + 1) * G].double().reshape(nq * G, D)
            o, e = _attend64(q, kv[0], kv[1], limit, D ** -0.5)
            out[r, :, h] = o.view(nq, G, D)
            lse[r, :, h] = e.view(nq, G)
    return {"out": out.view(-1, H, D), "lse": lse.view(-1, H) if case["lse"] else None}


def _exact_prompt(s):
    case = s["case"]
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    out = torch.empty((s["q"].shape[0], H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEV)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        q0, q1, k0, k1 = cq[b], cq[b + 1], ck[b], ck[b + 1]
        n, m = q1 - q0, k1 - k0
        limit = (torch.arange(n, device=DEV) + (m - n + 1)) if case["causal"] else torch.full((n,), m, device=DEV)
        for h in range(H):
            g = h * K // H
            o, e = _attend64(s["q"][q0:q1, h].double(), s["k"][k0:k1, g].double(), s["v"][k0:k1, g].double(), limit,
                             D ** -0.5)
            out[q0:q1, h] = o
            lse[q0:q1, h] = e
    return {"out": out, "lse": lse if case["lse"] else None}

"""Timed cases of the serving operators that follow the norm + quantisation ops:
slot maps, the paged NVFP4 cache (store and load), attention over it, and the
FP8 block-scaled matrix product.

``own = False`` computes every operator in plain torch; ``own = True`` makes
the calls of this package.  ``listed()`` names the cases, ``draw()`` gives
others of the same ranges, ``exact()`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# magnitudes of the E2M1 codes 0..7, and the midpoints between neighbours
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step of 64 running requests, captured into a graph: latency
        {"name": "slots_decode_64", "op": "slots", "requests": 64, "max_query": 1, "max_context": 8192, "page": 16,
         "pad": 0},
        # a large mixed step: most requests decode, some bring prompts; a padded token buffer
        {"name": "slots_mixed_1000", "op": "slots", "requests": 1000, "max_query": 300, "max_context": 30000, "page": 16,
         "pad": 77},
        # a decode step writes one token of each of 256 requests (Llama head layout) and reads them back
        {"name": "cache_decode_256", "op": "cache", "tokens": 256, "kv_heads": 8, "head_dim": 128, "page": 16,
         "dtype": "fp16", "pad": 0},
        # a prompt step, odd token count with padding (Qwen3 head layout)
        {"name": "cache_prompt_16001", "op": "cache", "tokens": 16001, "kv_heads": 4, "head_dim": 128, "page": 64,
         "dtype": "bf16", "pad": 30},
        # decode of a few short conversations: latency
        {"name": "attn_decode_short", "op": "attn", "requests": 8, "min_query": 1, "max_query": 1, "max_context": 500,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "bf16", "window": 0},
        # decode of an ordinary ragged batch (Qwen3 head layout)
        {"name": "attn_decode_ragged", "op": "attn", "requests": 128, "min_query": 1, "max_query": 1,
         "max_context": 8192, "heads": 32, "kv_heads": 4, "head_dim": 128, "page": 64, "dtype": "bf16", "window": 0},
        # decode of a few long documents: the keys have to be split over the card
        {"name": "attn_decode_long", "op": "attn", "requests": 3, "min_query": 1, "max_query": 1, "max_context": 131071,
         "heads": 64, "kv_heads": 8, "head_dim": 128, "page": 128, "dtype": "fp16", "window": 0},
        # prompts: two requests bring new tokens on top of cached ones
        {"name": "attn_prompt", "op": "attn", "requests": 2, "min_query": 1500, "max_query": 2500, "max_context": 2000,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "bf16", "window": 0},
        # a single decoded token through a square projection: latency
        {"name": "matmul_1x4096x4096", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "mode": "fp8_group128_row",
         "dtype": "bf16"},
        # an odd decode batch through the Llama down projection: bound by the weight's bytes
        {"name": "matmul_33x4096x14336", "op": "matmul", "m": 33, "n": 4096, "k": 14336,
         "mode": "fp8_group128_col+ue8m0+tma", "dtype": "bf16"},
        # a ragged prompt through the Llama QKV projection
        {"name": "matmul_1001x6144x4096", "op": "matmul", "m": 1001, "n": 6144, "k": 4096,
         "mode": "fp8_group128_col+tma", "dtype": "fp16"},
        # a full prefill step at the DeepSeek-V3 hidden size
        {"name": "matmul_8192x4096x7168", "op": "matmul", "m": 8192, "n": 4096, "k": 7168, "mode": "fp8_group128_row",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "cache", "attn", "attn", "matmul", "matmul"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "slots":
        requests = _log(rng, 1, 1000)
        return {"op": op, "requests": requests, "max_query": _log(rng, 1, 300), "max_context": _log(rng, 20, 30000),
                "page": page, "pad": rng.choice([0, 5, 77])}
    head_dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "cache":
        return {"op": op, "tokens": _log(rng, 1, 16001 * 4 * 128 // (kv_heads * head_dim)), "kv_heads": kv_heads,
                "head_dim": head_dim, "page": page, "dtype": dtype, "pad": rng.choice([0, 30])}
    if op == "attn":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16])
        window = rng.choice([0, 0, 0, 100, 1024])
        if rng.random() < 0.65:      # decode, some of it with a few speculative tokens
            requests = _log(rng, 1, 128)
            top = max(64, min(131071, 3 * 131071 * 8 * 128 // (requests * kv_heads * head_dim * 2)))
            return {"op": op, "requests": requests, "min_query": 1, "max_query": rng.choice([1, 1, 1, 4]),
                    "max_context": _log(rng, 20, top), "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
                    "page": page, "dtype": dtype, "window": window}
        requests = rng.randint(1, 3)
        # heads * head_dim at most 4096 and the keys of the listed prompts: no dearer than they are
        heads = min(heads, 4096 // head_dim // kv_heads * kv_heads)
        most = 5000 // requests
        new = _log(rng, 5, max(6, most // 2))
        return {"op": op, "requests": requests, "min_query": max(1, new // 2), "max_query": new,
                "max_context": rng.randint(1, max(2, most - new)), "heads": heads, "kv_heads": kv_heads,
                "head_dim": head_dim, "page": page, "dtype": dtype, "window": window}
    n, k = 8 * _log(rng, 16, 1800), 128 * _log(rng, 1, 112)
    m = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 7168 // (n * k))))
    return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype,
            "mode": rng.choice(["fp8_group128_row", "fp8_group128_col", "fp8_group128_col+tma", "fp8_group128_row+ue8m0",
                                "fp8_group128_col+ue8m0+tma"])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case, g, dev):
    """Query lengths and context lengths of the requests: ragged, the same
    lengths for every seed (so that outputs keep their shapes), in an order of
    the seed's."""
    R = case["requests"]
    lo, hi = case.get("min_query", 0), case["max_query"]
    rng = random.Random(R * 1000003 + hi)
    if case["op"] == "slots":       # nine in ten requests decode, the others bring up to max_query tokens
        q = [rng.randint(1, hi) if rng.random() < 0.1 else 1 for _ in range(R)]
    else:
        q = [rng.randint(lo, hi) for _ in range(R)]
    ctx = [rng.randint(case["max_context"] // 4, case["max_context"]) for _ in range(R)]
    order = torch.randperm(R, generator=g, device=dev)
    return torch.tensor(q, device=dev)[order], torch.tensor(ctx, device=dev)[order]


def _global_scale(x, g):
    """448 * 6 over a calibrated largest magnitude, a little above this data's own."""
    room = 1.03 + 0.1 * torch.rand((), generator=g, device=x.device)
    return (2688.0 / (x.float().abs().amax() * room)).reshape(1)


def _pages(lens, page, g, dev):
    """A shuffled page pool large enough for requests of `lens` tokens (host
    ints), and a block table that gives them its first pages."""
    need = [(n + page - 1) // page for n in lens]
    total, width = sum(need), max(1, max(need))
    pool = torch.randperm(total + 8, generator=g, device=dev).int()
    counts = torch.tensor(need, device=dev)
    start = counts.cumsum(0) - counts
    col = torch.arange(width, device=dev)
    table = pool[(start[:, None] + col).clamp(max=total + 7)]
    table = torch.where(col < counts[:, None], table, torch.full_like(table, -1))
    return table.contiguous(), pool, total


def _quant_rows(y, gs):
    """NVFP4 of the last axis in blocks of 16: packed codes and E4M3 scale bytes."""
    y = y.float()
    b = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    sb = (b.abs().amax(-1) / 6.0 * gs).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = sb.float()
    r = torch.where(d > 0, gs / d, torch.zeros_like(d))
    a = b * r[..., None]
    m = a.abs()
    # nearest code, ties to the even one
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(a)).to(torch.uint8).reshape(y.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb.view(torch.uint8)


def _values(codes, scales):
    """q * d of packed codes [.., D/2] and scale bytes [.., D/16] (exact in fp32)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    q = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    d = scales.view(torch.float8_e4m3fn).float()
    return (q.unflatten(-1, (-1, 16)) * d[..., None]).flatten(-2)


def _split(cache, page, D):
    """Views of a cache [pages, 2, heads, page*D*9/16]: codes [.., page, D/2] and scales [.., page, D/16]."""
    codes = cache[..., : page * D // 2].unflatten(-1, (page, D // 2))
    return codes, cache[..., page * D // 2:].unflatten(-1, (page, D // 16))


def _heads(shape, g, dev, outlier=4.0):
    """Normal keys / values with a few strong channels, as trained models have them."""
    x = torch.randn(shape, generator=g, device=dev)
    gain = torch.ones(shape[-1], device=dev)
    gain[torch.randperm(shape[-1], generator=g, device=dev)[:3]] = outlier
    return x * gain


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] == "slots":
        q, ctx = _lengths(case, g, dev)
        page = case["page"]
        table, pool, total = _pages((q + ctx).tolist(), page, g, dev)
        held = (ctx + page - 1) // page
        table = torch.where(torch.arange(table.shape[1], device=dev) < held[:, None], table, torch.full_like(table, -1))
        free = torch.randperm(pool.numel() + 1000, generator=g, device=dev).int()
        used = torch.zeros(free.numel(), dtype=torch.bool, device=dev)
        used[table[table >= 0].long()] = True
        free = free[~used[free.long()]]
        tokens = int(q.sum()) + case["pad"]
        return {"case": case, "query_lens": q.int(), "context_lens": ctx.int(), "table": table.contiguous(),
                "free": free.contiguous(), "num_free": torch.tensor([free.numel()], dtype=torch.int32, device=dev),
                "tokens": tokens}
    if case["op"] == "cache":
        n, nkv, D, page = case["tokens"], case["kv_heads"], case["head_dim"], case["page"]
        dt = DTYPES[case["dtype"]]
        k = _heads((n, nkv, D), g, dev).to(dt)
        v = _heads((n, nkv, D), g, dev, 2.0).to(dt)
        qkv = torch.cat([torch.randn(n, 4 * nkv * D, generator=g, device=dev).to(dt), k.flatten(1), v.flatten(1)], 1)
        pages = (n + page - 1) // page + 3
        slots = torch.randperm(pages * page, generator=g, device=dev)[:n]
        slots[n - min(case["pad"], n - 1):] = -1 if case["pad"] and n > 1 else slots[n - min(case["pad"], n - 1):]
        cache = torch.zeros(pages, 2, nkv, page * D * 9 // 16, dtype=torch.uint8, device=dev)
        return {"case": case, "qkv": qkv, "slots": slots, "k_gs": _global_scale(k, g), "v_gs": _global_scale(v, g),
                "cache": cache}
    if case["op"] == "attn":
        q_len, ctx = _lengths(case, g, dev)
        seq = (q_len + ctx).tolist()
        page, nkv, D = case["page"], case["kv_heads"], case["head_dim"]
        table, pool, total = _pages(seq, page, g, dev)
        cache = torch.empty(pool.numel(), 2, nkv, page * D * 9 // 16, dtype=torch.uint8, device=dev)
        codes, scales = _split(cache, page, D)
        gs = []
        for i in range(2):
            x = _heads((pool.numel(), nkv, page, D), g, dev, 4.0 if i == 0 else 2.0).to(DTYPES[case["dtype"]])
            gs.append(_global_scale(x, g))
            c, s = _quant_rows(x, gs[i])
            codes[:, i], scales[:, i] = c, s
        T = int(q_len.sum())
        q = torch.randn(T, case["heads"] * D, generator=g, device=dev).to(DTYPES[case["dtype"]])
        start = torch.zeros(case["requests"] + 1, dtype=torch.int32, device=dev)
        start[1:] = q_len.cumsum(0)
        return {"case": case, "q": q.view(T, case["heads"], D), "cache": cache, "table": table, "start": start,
                "seq": torch.tensor(seq, dtype=torch.int32, device=dev), "k_gs": gs[0], "v_gs": gs[1],
                "max_query": int(q_len.max()), "workspace": {}}
    m, n, k = case["m"], case["n"], case["k"]
    x = torch.randn(m, k, generator=g, device=dev)
    x[:, torch.randperm(k, generator=g, device=dev)[: max(1, k // 100)]] *= 20.0
    w = torch.randn(n, k, generator=g, device=dev) * 0.02
    amax = x.unflatten(1, (-1, 128)).abs().amax(-1)
    sa = (amax / 448.0).clamp(min=1e-12)
    if "ue8m0" in case["mode"]:
        sa = torch.exp2(torch.ceil(torch.log2(sa)))
    a_q = (x.unflatten(1, (-1, 128)) / sa[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    nb = (n + 127) // 128
    wp = torch.zeros(nb * 128, k, device=dev)
    wp[:n] = w
    blocks = wp.view(nb, 128, k // 128, 128)
    sb = (blocks.abs().amax((1, 3)) / 448.0).clamp(min=1e-12)
    b_q = (blocks / sb[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(nb * 128, k)[:n].contiguous()
    if "ue8m0" in case["mode"]:
        sa = ((sa.view(torch.int32) >> 23) & 255).to(torch.uint8)
    if "_col" in case["mode"]:
        per16 = 16 // sa.element_size()
        cols = (m + per16 - 1) // per16 * per16 if "tma" in case["mode"] else m
        col = torch.zeros(k // 128, cols, dtype=sa.dtype, device=dev)
        col[:, :m] = sa.t()
        sa = col
    return {"case": case, "a": a_q, "sa": sa.contiguous(), "b": b_q, "sb": sb.contiguous()}


# ---------------------------------------------------------------------------
# The passes
# ---------------------------------------------------------------------------
def _run_slots(s):
    c, page, tokens = s["case"], s["case"]["page"], s["tokens"]
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        slots, pos, start, seq, left, status = rq.build_slot_map(s["context_lens"], s["query_lens"], s["table"], s["free"],
                                                                 s["num_free"], page, tokens)
        return {"slots": slots, "positions": pos, "query_start": start, "seq_lens": seq, "num_free": left,
                "status": status, "table": s["table"]}
    q, ctx, table = s["query_lens"].long(), s["context_lens"].long(), s["table"]
    R, width = table.shape
    seq = q + ctx
    held, want = (ctx + page - 1) // page, (seq + page - 1) // page
    new = want - held
    before = new.cumsum(0) - new
    start = torch.zeros(R + 1, dtype=torch.int64, device=q.device)
    start[1:] = q.cumsum(0)
    bad = (new.sum() > s["num_free"].long()).int() + 2 * (want > width).any().int() + 4 * (start[-1:] > tokens).int()
    col = torch.arange(width, device=q.device)
    take = (s["num_free"].long() - 1 - before[:, None] - (col - held[:, None])).clamp(0, s["free"].numel() - 1)
    fresh = (col >= held[:, None]) & (col < want[:, None])
    table.copy_(torch.where(fresh, s["free"][take], table))
    tok = torch.arange(tokens, device=q.device)
    r = torch.searchsorted(start[1:].contiguous(), tok, right=True).clamp(max=R - 1)
    pos = ctx[r] + tok - start[r]
    live = tok < start[-1]
    slot = table[r, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    none = torch.full_like(tok, -1)
    return {"slots": torch.where(live, slot, none), "positions": torch.where(live, pos, none), "query_start": start.int(),
            "seq_lens": seq.int(), "num_free": (s["num_free"].long() - new.sum()).int(), "status": bad.int(),
            "table": table}


def _run_cache(s):
    c = s["case"]
    n, nkv, D, page = c["tokens"], c["kv_heads"], c["head_dim"], c["page"]
    k = s["qkv"][:, 4 * nkv * D: 5 * nkv * D].unflatten(1, (nkv, D))
    v = s["qkv"][:, 5 * nkv * D:].unflatten(1, (nkv, D))
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        rq.kv_cache_store_nvfp4(k, v, s["slots"], s["k_gs"], s["v_gs"], s["cache"], page)
        k2, v2 = rq.kv_cache_load_nvfp4(s["cache"], s["slots"], s["k_gs"], s["v_gs"], D, page, k.dtype)
        return {"k": k2, "v": v2}
    codes, scales = _split(s["cache"], page, D)
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    p, i = at // page, at % page
    out = {}
    kept = torch.where(live, at, at.new_full((), s["cache"].shape[0] * page))
    for side, (name, x, gs) in enumerate((("k", k, s["k_gs"]), ("v", v, s["v_gs"]))):
        cq, sq = _quant_rows(x, gs)
        # padding rows go to a row behind the last slot, which is dropped
        for part, rows in ((codes, cq), (scales, sq)):
            flat = part[:, side].transpose(1, 2).flatten(0, 1)
            flat = torch.cat([flat, flat[:1]])
            flat[kept] = rows
            part[:, side] = flat[:-1].unflatten(0, (-1, page)).transpose(1, 2)
        y = _values(codes[p, side, :, i], scales[p, side, :, i]) / gs
        out[name] = torch.where(live[:, None, None], y, torch.zeros_like(y)).to(x.dtype)
    return out


def _run_attn(s):
    c = s["case"]
    D, page, nkv = c["head_dim"], c["page"], c["kv_heads"]
    scale = 1.0 / math.sqrt(D)
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        if "buffer" not in s["workspace"]:
            size = rq.paged_attention_workspace_bytes(s["q"].shape[0], c["requests"], c["heads"], nkv, D)
            s["workspace"]["buffer"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        out, lse = rq.paged_attention_nvfp4(s["q"], s["cache"], s["table"], s["start"], s["seq"], s["k_gs"], s["v_gs"], page,
                                            scale, window=c["window"], return_lse=True,
                                            workspace=s["workspace"]["buffer"])
        return {"out": out, "lse": lse}
    codes, scales = _split(s["cache"], page, D)
    table = s["table"].clamp(min=0).long()
    R, L, G = c["requests"], table.shape[1] * page, c["heads"] // nkv
    T, Q = s["q"].shape[0], s["max_query"]
    k, v = ((_values(codes[table, i], scales[table, i]) / s[gs]).transpose(2, 3).reshape(R, L, nkv, D)
            for i, gs in ((0, "k_gs"), (1, "v_gs")))
    start, seq = s["start"].long(), s["seq"].long()
    i = torch.arange(Q, device=k.device)
    q_len = start[1:] - start[:-1]
    rows = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[rows].view(R, Q, nkv, G, D)
    logits = torch.einsum("rqhgd,rlhd->rhgql", q, k) * scale
    pos = (seq - q_len)[:, None] + i                       # [R, Q]
    key = torch.arange(L, device=k.device)
    ok = (key <= pos[..., None]) & (key < seq[:, None, None])
    if c["window"]:
        ok &= key > pos[..., None] - c["window"]
    logits = logits.masked_fill(~ok[:, None, None], float("-inf"))
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("rhgql,rlhd->rqhgd", e / total.clamp(min=1e-30), v)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    live = (i < q_len[:, None]).flatten().nonzero().squeeze(1) if Q > 1 else torch.arange(R, device=k.device)
    return {"out": out.reshape(R * Q, c["heads"], D)[live].to(s["q"].dtype),
            "lse": lse.reshape(R * Q, c["heads"])[live].float()}


def _run_matmul(s):
    c = s["case"]
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        return rq.fp8_block_matmul(s["a"], s["sa"], c["mode"], s["b"], s["sb"], DTYPES[c["dtype"]])
    sa = s["sa"]
    if "ue8m0" in c["mode"]:
        sa = torch.exp2(sa.float() - 127.0)
    if "_col" in c["mode"]:
        sa = sa[:, : c["m"]].t()
    a = (s["a"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * sa[..., None]).flatten(1)
    sb = s["sb"].repeat_interleave(128, 0)[: c["n"]]
    b = (s["b"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * sb[..., None]).flatten(1)
    return (a @ b.t()).to(DTYPES[c["dtype"]])


def run(state):
    return {"slots": _run_slots, "cache": _run_cache, "attn": _run_attn, "matmul": _run_matmul}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "slots":
        # expected tokens: nine in ten requests bring one, the others half of max_query
        R = case["requests"]
        tokens = R * (0.9 + 0.1 * (1 + case["max_query"]) / 2) + case["pad"]
        return {"bytes": int(R * 20 + tokens * 16 + tokens / case["page"] * 8), "flops": int(tokens * 6 + R * 8)}
    if case["op"] == "cache":
        e = case["tokens"] * case["kv_heads"] * case["head_dim"] * 2       # elements of K and V
        return {"bytes": int(e * 2 + 2 * e * 9 / 16 + e * 2 + case["tokens"] * 16), "flops": e * 6}
    if case["op"] == "attn":
        R, nkv, D, H = case["requests"], case["kv_heads"], case["head_dim"], case["heads"]
        q = (case["min_query"] + case["max_query"]) / 2
        ctx = 0.625 * case["max_context"]
        keys = min(ctx + q, case["window"] + q) if case["window"] else ctx + q
        seen = min(ctx + (q + 1) / 2, case["window"]) if case["window"] else ctx + (q + 1) / 2
        return {"bytes": int(R * keys * nkv * D * 9 / 8 + R * q * H * (4 * D + 4)), "flops": int(4 * D * H * R * q * seen)}
    m, n, k = case["m"], case["n"], case["k"]
    width = 1 if "ue8m0" in case["mode"] else 4
    return {"bytes": m * k + n * k + 2 * m * n + m * k // 128 * width + (n + 127) // 128 * (k // 128) * 4,
            "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_round_e2m1(a):
    grid = torch.tensor(E2M1, dtype=torch.float64, device=a.device)
    m = a.abs().clamp(max=6.0)
    hi = torch.searchsorted(grid, m).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = m - grid[lo], grid[hi] - m
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[pick], a)


def _exact_round_e4m3(x):
    """Nearest E4M3 value of non-negative x (even fraction on ties), at most 448."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** -9))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _exact_cache(s):
    c = s["case"]
    nkv, D = c["kv_heads"], c["head_dim"]
    out = {}
    for at, name in ((4, "k"), (5, "v")):
        y = s["qkv"][:, at * nkv * D: (at + 1) * nkv * D].double().reshape(c["tokens"], nkv, D // 16, 16)
        gs = s[name + "_gs"].double()
        d = _exact_round_e4m3(y.abs().amax(-1, keepdim=True) / 6 * gs)
        q = _exact_round_e2m1(torch.where(d > 0, y * gs / d.clamp(min=1e-300), torch.zeros_like(y)))
        out[name] = (q * d / gs).reshape(c["tokens"], nkv, D) * (s["slots"] >= 0)[:, None, None]
    return out


def _exact_attn(s):
    c = s["case"]
    D, page, nkv, H = c["head_dim"], c["page"], c["kv_heads"], c["heads"]
    start, seq = s["start"].tolist(), s["seq"].tolist()
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=s["q"].device)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=s["q"].device)
    outs, lses = [], []
    for r in range(c["requests"]):
        n = seq[r]
        raw = s["cache"][s["table"][r, : (n + page - 1) // page].long()]       # [pages, 2, heads, bytes]
        kv = []
        for i, gs in ((0, s["k_gs"]), (1, s["v_gs"])):
            bytes_ = raw[:, i, :, : page * D // 2].reshape(-1, nkv, page, D // 2, 1)
            nib = torch.cat([bytes_ & 15, bytes_ >> 4], -1).reshape(-1, nkv, page, D // 16, 16).long()
            d = raw[:, i, :, page * D // 2:].reshape(-1, nkv, page, D // 16, 1)
            x = grid[nib & 7] * sign[nib >> 3] * d.view(torch.float8_e4m3fn).double() / gs.double()
            kv.append(x.permute(1, 0, 2, 3, 4).reshape(nkv, -1, D)[:, :n])
        q = s["q"][start[r]: start[r + 1]].double()
        m = q.shape[0]
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        key = torch.arange(n, device=q.device)[None]
        ok = key <= pos
        if c["window"]:
            ok = ok & (key > pos - c["window"])
        out = torch.empty(m, H, D, dtype=torch.float64, device=q.device)
        lse = torch.empty(m, H, dtype=torch.float64, device=q.device)
        for h in range(nkv):
            hs = slice(h * (H // nkv), (h + 1) * (H // nkv))
            z = (q[:, hs].transpose(0, 1) @ kv[0][h].t()) / math.sqrt(D)
            z = torch.where(ok, z, torch.full_like(z, -math.inf))
            out[:, hs] = (torch.softmax(z, -1) @ kv[1][h]).transpose(0, 1)
            lse[:, hs] = torch.logsumexp(z, -1).t()
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_matmul(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    sa = s["sa"].double()
    if "ue8m0" in c["mode"]:
        sa = torch.pow(2.0, sa - 127)
    if "_col" in c["mode"]:
        sa = sa[:, :m].transpose(0, 1)
    out = torch.zeros(m, n, dtype=torch.float64, device=sa.device)
    block = torch.arange(n, device=sa.device) // 128
    for b in range(k // 128):
        cols = slice(b * 128, (b + 1) * 128)
        part = s["a"][:, cols].view(torch.float8_e4m3fn).double() @ s["b"][:, cols].view(torch.float8_e4m3fn).double().t()
        out += part * sa[:, b, None] * s["sb"].double()[block, b]
    return out


def exact(case, seed):
    if case["op"] == "slots":
        return None          # whole numbers: compared as they are
    return {"cache": _exact_cache, "attn": _exact_attn, "matmul": _exact_matmul}[case["op"]](prepare(case, seed))

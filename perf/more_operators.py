"""Timed cases of the attention path over an 8-bit cache: QK-norm + rotary
positions with three axes (time, height, width), the paged FP8 cache with a
power-of-two scale per block of 16 tokens and head (store and load), and
attention over it.

``own = False`` computes every operator in plain torch; ``own = True`` makes
the calls of this package.  ``listed()`` names the cases, ``draw()`` gives
others of the same ranges, ``exact()`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16              # tokens that share a scale
LEAST = -39             # exponent of the smallest scale: that of the library's floor 1e-12, rounded up
MAX_POSITIONS = 32768


def listed():
    return [
        # one decode step of 64 conversations about images: latency
        {"name": "mrope_decode_64", "op": "mrope", "tokens": 64, "q_heads": 32, "kv_heads": 4, "head_dim": 128,
         "t": 24, "h": 20, "w": 20, "interleaved": True, "neox": True, "norm": True, "dtype": "bf16", "pad": 0},
        # frames of a video in an odd number of tokens, no norm, axes one after the other, padded token buffer
        {"name": "mrope_video_2001", "op": "mrope", "tokens": 2001, "q_heads": 28, "kv_heads": 4, "head_dim": 128,
         "t": 16, "h": 24, "w": 24, "interleaved": False, "neox": True, "norm": False, "dtype": "fp16", "pad": 47},
        # a prefill step of text and images (Qwen3 head layout)
        {"name": "mrope_images_16384", "op": "mrope", "tokens": 16384, "q_heads": 32, "kv_heads": 4, "head_dim": 128,
         "t": 24, "h": 20, "w": 20, "interleaved": True, "neox": True, "norm": True, "dtype": "bf16", "pad": 0},
        # a decode step writes one token of each of 256 requests into blocks that are partly filled (Llama head layout)
        {"name": "cache8_decode_256", "op": "cache", "requests": 256, "min_query": 1, "max_query": 1, "max_context": 2000,
         "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "fp16", "pad": 0},
        # three prompts behind cached prefixes of odd lengths, with padding (Qwen3 head layout)
        {"name": "cache8_prompt_16000", "op": "cache", "requests": 3, "min_query": 5000, "max_query": 6001,
         "max_context": 777, "kv_heads": 4, "head_dim": 128, "page": 64, "dtype": "bf16", "pad": 30},
        # decode of a few short conversations: latency
        {"name": "attn8_decode_short", "op": "attn", "requests": 8, "prompts": 0, "min_query": 1, "max_query": 1,
         "max_context": 500, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "bf16", "window": 0},
        # decode of an ordinary ragged batch (Qwen3 head layout)
        {"name": "attn8_decode_ragged", "op": "attn", "requests": 128, "prompts": 0, "min_query": 1, "max_query": 1,
         "max_context": 8192, "heads": 32, "kv_heads": 4, "head_dim": 128, "page": 64, "dtype": "bf16", "window": 0},
        # decode of a few long documents: the keys have to be split over the card
        {"name": "attn8_decode_long", "op": "attn", "requests": 3, "prompts": 0, "min_query": 1, "max_query": 1,
         "max_context": 131071, "heads": 64, "kv_heads": 8, "head_dim": 128, "page": 128, "dtype": "fp16", "window": 0},
        # four speculative tokens a request, small heads in an odd group, a sliding window
        {"name": "attn8_window_spec", "op": "attn", "requests": 33, "prompts": 0, "min_query": 4, "max_query": 4,
         "max_context": 6000, "heads": 15, "kv_heads": 3, "head_dim": 64, "page": 32, "dtype": "fp16", "window": 1000},
        # decode with heads of 256
        {"name": "attn8_head256", "op": "attn", "requests": 48, "prompts": 0, "min_query": 1, "max_query": 1,
         "max_context": 4096, "heads": 16, "kv_heads": 2, "head_dim": 256, "page": 64, "dtype": "bf16", "window": 0},
        # prompts: two requests bring new tokens on top of cached ones
        {"name": "attn8_prompt", "op": "attn", "requests": 2, "prompts": 2, "min_query": 1500, "max_query": 2500,
         "max_context": 2000, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "bf16", "window": 0},
        # a chunk of a prompt beside running requests
        {"name": "attn8_mixed", "op": "attn", "requests": 24, "prompts": 1, "min_query": 1, "max_query": 509,
         "max_context": 1500, "heads": 16, "kv_heads": 4, "head_dim": 128, "page": 16, "dtype": "bf16", "window": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mrope", "mrope", "cache", "cache", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    head_dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if op == "mrope":
        q_heads = kv_heads * rng.choice([1, 2, 3, 5, 8])
        interleaved = rng.random() < 0.5
        if interleaved:         # height and width take every third angle up to their sections' ends
            h, w = rng.randint(0, head_dim // 6), rng.randint(0, head_dim // 6)
        elif rng.random() < 0.5:
            h, w = 4 * rng.randint(0, head_dim // 32), 4 * rng.randint(0, head_dim // 16 // 2)
        else:
            h, w = rng.randint(0, head_dim // 6), rng.randint(0, head_dim // 6)
        return {"op": op, "tokens": _log(rng, 1, 16384 * 38 * 128 // ((q_heads + kv_heads + 2) * head_dim)),
                "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "t": head_dim // 2 - h - w, "h": h, "w": w,
                "interleaved": interleaved, "neox": rng.random() < 0.7, "norm": rng.random() < 0.7, "dtype": dtype,
                "pad": rng.choice([0, 0, 9])}
    if op == "cache":
        most = 16000 * 4 * 128 // (kv_heads * head_dim)
        requests = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, most // requests))
        return {"op": op, "requests": requests, "min_query": max(1, new // 2), "max_query": new,
                "max_context": rng.randint(1, 2000), "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
                "dtype": dtype, "pad": rng.choice([0, 30])}
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16])
    window = rng.choice([0, 0, 0, 100, 1024])
    if rng.random() < 0.6:      # decode, some of it with a few speculative tokens
        requests = _log(rng, 1, 128)
        top = max(64, min(131071, 3 * 131071 * 8 * 128 // (requests * kv_heads * head_dim * 2)))
        new = rng.choice([1, 1, 1, 4])
        return {"op": op, "requests": requests, "prompts": 0, "min_query": new, "max_query": new,
                "max_context": _log(rng, 20, top), "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
                "dtype": dtype, "window": window}
    # prompts, alone or beside a few decodes; heads * head_dim and the keys no dearer than the listed prompts'
    requests = rng.randint(1, 3)
    heads = max(kv_heads, min(heads, 4096 // head_dim // kv_heads * kv_heads))
    most = 5000 // requests
    new = _log(rng, 5, max(6, most // 2))
    return {"op": op, "requests": requests, "prompts": rng.randint(1, requests), "min_query": max(1, new // 2),
            "max_query": new, "max_context": rng.randint(1, max(2, most - new)), "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "dtype": dtype, "window": window}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case, g, dev):
    """Query and context lengths of the requests: ragged, the same ones for
    every seed (so that outputs keep their shapes), in an order of the seed's."""
    R, lo, hi = case["requests"], case["min_query"], case["max_query"]
    prompts = case.get("prompts", R) or R
    rng = random.Random(R * 1000003 + hi)
    q = [rng.randint(lo, hi) if r < prompts else 1 for r in range(R)]
    ctx = [rng.randint(case["max_context"] // 4, case["max_context"]) for _ in range(R)]
    order = torch.randperm(R, generator=g, device=dev)
    return torch.tensor(q, device=dev)[order], torch.tensor(ctx, device=dev)[order]


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
    return table.contiguous(), pool


def _heads(shape, g, dev, outlier):
    """Normal keys / values with a few strong channels and tokens of different strength."""
    x = torch.randn(shape, generator=g, device=dev)
    gain = torch.ones(shape[-1], device=dev)
    gain[torch.randperm(shape[-1], generator=g, device=dev)[:3]] = outlier
    return x.mul_(gain).mul_(0.5 + 1.5 * torch.rand(*shape[:-1], 1, generator=g, device=dev))


def _exponent(amax):
    """Exponent of the smallest power of two s with amax / s <= 448."""
    m, e = torch.frexp(amax / 448.0)
    return torch.where(m == 0.5, e - 1, e).clamp(min=LEAST)


def _filled_cache(pages, nkv, page, D, g, dev, dtype):
    """A cache whose every block holds 16 tokens as the store would have written them."""
    codes = torch.empty(pages, 2, nkv, page, D, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, 2, nkv, page // BLOCK, dtype=torch.uint8, device=dev)
    for side, outlier in ((0, 4.0), (1, 2.0)):
        x = _heads((pages, nkv, page, D), g, dev, outlier).to(dtype).float()
        e = _exponent(x.unflatten(2, (-1, BLOCK)).abs().amax((-1, -2)))
        x = torch.ldexp(x, -e.repeat_interleave(BLOCK, -1)[..., None])
        codes[:, side] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[:, side] = (e + 127).to(torch.uint8)
    return codes, scales


def _positions(n, g, dev):
    """Positions of text and of images in it: where a token is part of an image
    its time stands still while height and width walk the image."""
    at = torch.arange(n, device=dev) + torch.randint(0, MAX_POSITIONS // 2 - n if n < MAX_POSITIONS // 2 else 1, (1,),
                                                     generator=g, device=dev)
    at = at % (MAX_POSITIONS - 64)
    image = (torch.arange(n, device=dev) // 600) % 2 == 1
    inside = torch.arange(n, device=dev) % 600
    base = at - inside
    pos = torch.stack([at, at, at])
    pos[0] = torch.where(image, base, pos[0])
    pos[1] = torch.where(image, base + inside // 30, pos[1])
    pos[2] = torch.where(image, base + inside % 30, pos[2])
    return pos.clamp(min=0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    D, nkv = case["head_dim"], case["kv_heads"]
    if case["op"] == "mrope":
        n, nq = case["tokens"], case["q_heads"]
        qkv = torch.randn(n, (nq + 2 * nkv) * D, generator=g, device=dev).to(dt)
        pos = _positions(n, g, dev)
        pad = min(case["pad"], n - 1)
        pos[:, n - pad:] = -1
        freq = torch.pow(1e6, -torch.arange(D // 2, device=dev, dtype=torch.float64) / (D // 2))
        angle = torch.arange(MAX_POSITIONS, device=dev, dtype=torch.float64)[:, None] * freq
        table = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        q_w, k_w = ((1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt) for _ in range(2))
        return {"case": case, "qkv": qkv, "pos": pos.contiguous(), "table": table, "q_w": q_w, "k_w": k_w,
                "out": torch.zeros(n, (nq + nkv) * D, dtype=dt, device=dev)}
    page = case["page"]
    q_len, ctx = _lengths(case, g, dev)
    seq = q_len + ctx
    table, pool = _pages(seq.tolist(), page, g, dev)
    cache, scales = _filled_cache(pool.numel(), nkv, page, D, g, dev, dt)
    T = int(q_len.sum())
    start = torch.zeros(case["requests"] + 1, dtype=torch.int32, device=dev)
    start[1:] = q_len.cumsum(0)
    if case["op"] == "cache":
        r = torch.repeat_interleave(torch.arange(case["requests"], device=dev), q_len)

        def slots(req, pos):
            return table[req, pos // page].long() * page + pos % page

        pos = ctx[r] + torch.arange(T, device=dev) - start[r].long()
        n = T + case["pad"]
        slot_map = torch.full((n,), -1, dtype=torch.int64, device=dev)
        slot_map[:T] = slots(r, pos)
        # what the step writes or rounds anew: from the first touched block of each request to its last token
        first = ctx // BLOCK * BLOCK
        count = seq - first
        rr = torch.repeat_interleave(torch.arange(case["requests"], device=dev), count)
        off = torch.arange(int(count.sum()), device=dev) - (count.cumsum(0) - count)[rr]
        k = _heads((n, nkv, D), g, dev, 4.0).to(dt)
        v = _heads((n, nkv, D), g, dev, 2.0).to(dt)
        qkv = torch.cat([torch.randn(n, 4 * nkv * D, generator=g, device=dev).to(dt), k.flatten(1), v.flatten(1)], 1)
        return {"case": case, "qkv": qkv, "slots": slot_map, "read": slots(rr, first[rr] + off), "cache": cache,
                "scales": scales}
    q = torch.randn(T, case["heads"], D, generator=g, device=dev).to(dt)
    return {"case": case, "q": q, "cache": cache, "scales": scales, "table": table, "start": start, "seq": seq.int(),
            "max_query": int(q_len.max()), "workspace": {}}


# ---------------------------------------------------------------------------
# The passes
# ---------------------------------------------------------------------------
def _axes(case, dev):
    """Axis (0 time, 1 height, 2 width) of each angle."""
    i = torch.arange(case["head_dim"] // 2, device=dev)
    if case["interleaved"]:
        h = (i % 3 == 1) & (i < 3 * case["h"])
        w = (i % 3 == 2) & (i < 3 * case["w"])
    else:
        h = (i >= case["t"]) & (i < case["t"] + case["h"])
        w = i >= case["t"] + case["h"]
    return h.long() + 2 * w.long()


def _run_mrope(s):
    c = s["case"]
    nq, nkv, D, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["tokens"]
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        q_w, k_w = (s["q_w"], s["k_w"]) if c["norm"] else (None, None)
        return rq.qk_norm_mrope(s["qkv"], s["pos"], s["table"], q_w, k_w, 1e-6, nq, nkv, D, (c["t"], c["h"], c["w"]),
                                c["neox"], interleaved=c["interleaved"], out=s["out"])
    x = s["qkv"][:, : (nq + nkv) * D].float().unflatten(1, (nq + nkv, D))
    if c["norm"]:
        w = torch.cat([s["q_w"].float().expand(nq, D), s["k_w"].float().expand(nkv, D)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    row = s["pos"].clamp(min=0)[_axes(c, x.device)].t()             # [n, D / 2]
    i = torch.arange(D // 2, device=x.device)
    cos, sin = s["table"][row, i][:, None], s["table"][row, D // 2 + i][:, None]
    if c["neox"]:
        a, b = x[..., : D // 2], x[..., D // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    live = (s["pos"] >= 0).all(0)[:, None]
    s["out"].copy_(torch.where(live, y.flatten(1).to(s["out"].dtype), s["out"]))
    return s["out"]


def _kv(s):
    c = s["case"]
    w = c["kv_heads"] * c["head_dim"]
    return (s["qkv"][:, i * w: (i + 1) * w].unflatten(1, (c["kv_heads"], c["head_dim"])) for i in (4, 5))


def _flat(codes, side):
    """Codes of a side as [heads, slots, D] (a copy)."""
    return codes[:, side].transpose(0, 1).flatten(1, 2)


def _run_cache(s):
    c = s["case"]
    k, v = _kv(s)
    if own:
        import residual_add_rmsnorm_rmsq_gb300 as rq
        rq.kv_cache_store_fp8(k, v, s["slots"], s["cache"], s["scales"])
        k2, v2 = rq.kv_cache_load_fp8(s["cache"], s["scales"], s["read"], k.dtype)
        return {"k": k2, "v": v2}
    nkv, D, page = c["kv_heads"], c["head_dim"], c["page"]
    live = (s["slots"] >= 0).nonzero().squeeze(1)
    slot = s["slots"][live]
    block, run, = torch.unique_consecutive(slot // BLOCK, return_inverse=True)
    head = torch.zeros_like(block).scatter_reduce_(0, run, slot % BLOCK, "amin", include_self=False)
    p, b = block // (page // BLOCK), block % (page // BLOCK)
    at = block[:, None] * BLOCK + torch.arange(BLOCK, device=slot.device)       # slots of the touched blocks
    for side, x in enumerate((k, v)):
        x = x[live].float()
        amax = torch.zeros(block.numel(), nkv, device=x.device).index_reduce_(0, run, x.abs().amax(-1), "amax")
        old = s["scales"][p, side, :, b].long() - 127
        e = _exponent(amax).long()
        e = torch.where(head[:, None] > 0, torch.maximum(e, old), e)
        codes = s["cache"][at // page, side, :, at % page].view(torch.float8_e4m3fn).float()     # [blocks, 16, heads, D]
        shift = torch.where(head[:, None] > 0, old - e, torch.zeros_like(e))
        codes = torch.ldexp(codes, shift[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        new = torch.ldexp(x, -e[run][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = codes.index_put((run, slot % BLOCK), new)
        s["cache"][at // page, side, :, at % page] = codes
        s["scales"][p, side, :, b] = (e + 127).to(torch.uint8)
    read, out = s["read"], {}
    for side, name in enumerate(("k", "v")):
        y = s["cache"][read // page, side, :, read % page].view(torch.float8_e4m3fn).float()
        e = s["scales"][read // page, side, :, read % page // BLOCK].long() - 127
        out[name] = torch.ldexp(y, e[..., None]).to(k.dtype)
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
        out, lse = rq.paged_attention_fp8(s["q"], s["cache"], s["scales"], s["table"], s["start"], s["seq"], scale,
                                          window=c["window"], return_lse=True, workspace=s["workspace"]["buffer"])
        return {"out": out, "lse": lse}
    table = s["table"].clamp(min=0).long()
    R, L, G = c["requests"], table.shape[1] * page, c["heads"] // nkv
    T, Q = s["q"].shape[0], s["max_query"]
    value = torch.exp2(s["scales"].float() - 127.0)
    k, v = ((s["cache"][table, i].view(torch.float8_e4m3fn).float() *
             value[table, i].repeat_interleave(BLOCK, -1)[..., None]).transpose(2, 3).reshape(R, L, nkv, D) for i in (0, 1))
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


def run(state):
    return {"mrope": _run_mrope, "cache": _run_cache, "attn": _run_attn}[state["case"]["op"]](state)


def _mean_lengths(case):
    """Mean number of new tokens, and of cached ones, of a request."""
    R, mid = case["requests"], (case["min_query"] + case["max_query"]) / 2
    prompts = case.get("prompts", R) or R
    return (mid * prompts + R - prompts) / R, 0.625 * case["max_context"]


def work(case):
    D = case["head_dim"]
    if case["op"] == "mrope":
        n, heads = case["tokens"], case["q_heads"] + case["kv_heads"]
        return {"bytes": int(n * (heads * D * 4 + D * 4 + 24)), "flops": int(n * heads * D * (7 if case["norm"] else 3))}
    nkv, R = case["kv_heads"], case["requests"]
    new, ctx = _mean_lengths(case)
    if case["op"] == "cache":
        e = 2 * nkv * D                 # elements of a token
        touched = R * (new + 7.5)       # 7.5 older tokens in the first block, on average
        return {"bytes": int(R * new * e * 3 + touched * e * 3 + (R * new + touched) * 8), "flops": int(R * new * e * 4)}
    H, w = case["heads"], case["window"]
    total = seen = 0.0
    mid = (case["min_query"] + case["max_query"]) / 2
    prompts = case["prompts"] or R
    for count, q in ((prompts, mid), (R - prompts, 1.0)):
        total += count * (min(ctx + q, w + q) if w else ctx + q)
        seen += count * q * (min(ctx + (q + 1) / 2, w) if w else ctx + (q + 1) / 2)
    return {"bytes": int(total * nkv * 2 * (D + 1 / BLOCK) + R * new * H * (4 * D + 4)), "flops": int(4 * D * H * seen)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_mrope(s):
    c = s["case"]
    nq, nkv, D, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["tokens"]
    pos = s["pos"]
    out = torch.zeros(n, nq + nkv, D, dtype=torch.float64, device=pos.device)
    x = s["qkv"].double().view(n, nq + 2 * nkv, D)[:, : nq + nkv]
    if c["norm"]:
        mean = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D
        x = x / torch.sqrt(mean + 1e-6)
        x = torch.cat([x[:, :nq] * s["q_w"].double(), x[:, nq:] * s["k_w"].double()], 1)
    for i in range(D // 2):
        if c["interleaved"]:
            axis = 1 if i % 3 == 1 and i < 3 * c["h"] else 2 if i % 3 == 2 and i < 3 * c["w"] else 0
        else:
            axis = 0 if i < c["t"] else 1 if i < c["t"] + c["h"] else 2
        at = pos[axis].clamp(min=0)
        turn = torch.complex(s["table"][at, i].double(), s["table"][at, D // 2 + i].double())[:, None]
        one, two = (i, i + D // 2) if c["neox"] else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., one], x[..., two]) * turn
        out[..., one], out[..., two] = z.real, z.imag
    return (out * (pos.amin(0) >= 0)[:, None, None]).flatten(1)


def _nearest_e4m3(x):
    """Nearest E4M3 value, even fraction on ties."""
    m = x.abs()
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -12))).clamp(min=-6) - 3)
    return torch.copysign((torch.round(m / step) * step).clamp(max=448.0), x)


def _e4m3_value(code):
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(c > 127, -v, v)


def _exact_cache(s):
    c = s["case"]
    page, dev = c["page"], s["qkv"].device
    slots = s["slots"][s["slots"] >= 0]
    total = s["cache"].shape[0] * page
    place = torch.full((total,), -1, dtype=torch.int64, device=dev)     # the new token of a slot
    place[slots] = torch.arange(slots.numel(), device=dev)
    groups = place.view(-1, BLOCK)
    first = (groups >= 0).long().argmax(1)                              # offset of a block's first new token
    block = s["read"] // BLOCK
    token = place[s["read"]]
    out = {}
    for side, (name, x) in enumerate(zip(("k", "v"), _kv(s))):
        x = x.double()
        amax = torch.zeros(total // BLOCK, c["kv_heads"], dtype=torch.float64, device=dev)
        amax.index_reduce_(0, slots // BLOCK, x[: slots.numel()].abs().amax(-1), "amax")
        least = torch.exp2(torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** LEAST))))
        # (log2 of a power of two may be off by its rounding)
        least = torch.where(least / 2 * 448 >= amax.clamp(min=448 * 2.0 ** LEAST), least / 2, least)
        old = torch.exp2(s["scales"][:, side].transpose(1, 2).reshape(-1, c["kv_heads"]).double() - 127)
        scale = torch.where(first[:, None] > 0, torch.maximum(least, old), least)
        kept = _e4m3_value(s["cache"][:, side].transpose(1, 2).reshape(total, c["kv_heads"], -1)[s["read"]])
        kept = kept * old[block][..., None]
        want = torch.where((token >= 0)[:, None, None], x[token.clamp(min=0)], kept)
        out[name] = _nearest_e4m3(want / scale[block][..., None]) * scale[block][..., None]
    return out


def _exact_attn(s):
    c = s["case"]
    D, page, nkv, H = c["head_dim"], c["page"], c["kv_heads"], c["heads"]
    start, seq = s["start"].tolist(), s["seq"].tolist()
    outs, lses = [], []
    for r in range(c["requests"]):
        n = seq[r]
        pages = s["table"][r, : (n + page - 1) // page].long()
        kv = []
        for side in (0, 1):
            x = _e4m3_value(s["cache"][pages, side])                    # [pages, heads, page, D]
            e = s["scales"][pages, side].double() - 127
            x = x.unflatten(2, (-1, BLOCK)) * torch.exp2(e)[..., None, None]
            kv.append(x.flatten(2, 3).transpose(0, 1).reshape(nkv, -1, D)[:, :n])
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


def exact(case, seed):
    return {"mrope": _exact_mrope, "cache": _exact_cache, "attn": _exact_attn}[case["op"]](prepare(case, seed))

"""Attention over the paged NVFP4 cache on the GPU, against float64 with
tolerances derived beside the reference (tests/_serve_ref.py)."""
import numpy as np
import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(q_lens, seq_lens, heads, kv, D, page, dtype, *, seed=0, extra_rows=0, sigma=1.0, spare=3):
    rng = np.random.default_rng(seed)
    need = [max(1, -(-s // page)) for s in seq_lens]
    pages, width = sum(need) + spare, max(need) + 1
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(seq_lens), width), -1, np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at: at + m]
        at += m
    cache = ref.random_cache(rng, pages, kv, page, D)
    T = sum(q_lens) + extra_rows
    q, q64 = ref.act(rng.normal(0, sigma, (T, heads, D)), DT[dtype])
    return {"q": q, "q64": q64, "cache": cache, "table": table, "q_lens": q_lens, "seq": seq_lens, "page": page, "D": D,
            "heads": heads, "kv": kv, "dtype": dtype, "k_gs": np.float32(611.3), "v_gs": np.float32(57.9)}


VARIANTS = ("direct", "pipelined")


def run(rq, c, *, window=0, scale=None, stream=None, **kw):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    start = np.concatenate([[0], np.cumsum(c["q_lens"])]).astype(np.int32)
    return rq.paged_attention_nvfp4(kw.pop("q", c["q"].cuda()), dev(c["cache"]), dev(c["table"]), dev(start),
                                    dev(np.array(c["seq"], np.int32)), torch.tensor([c["k_gs"]], device="cuda"),
                                    torch.tensor([c["v_gs"]], device="cuda"), c["page"], scale, window=window,
                                    return_lse=True, stream=stream, **kw)


def check(rq, c, *, window=0, scale=None, **kw):
    n = sum(c["q_lens"])
    out, lse = run(rq, c, window=window, scale=scale, **kw)
    eps = torch.finfo(DT[c["dtype"]]).eps
    w_out, w_lse, tol, tol_lse = ref.attention(c["q64"][:n], c["cache"], c["table"], c["q_lens"], c["seq"],
                                               float(c["k_gs"]), float(c["v_gs"]), c["page"],
                                               c["D"] ** -0.5 if scale is None else scale, window, eps)
    o, s = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    empty = np.isinf(w_lse)
    assert np.array_equal(np.isinf(s), empty) and (s[empty] < 0).all() and (o[empty] == 0).all()
    bad = np.abs(o - w_out) - tol
    assert bad.max(initial=0) <= 0, f"out off by up to {np.abs(o - w_out).max()}, {(bad > 0).sum()} beyond"
    bad = np.abs(s[~empty] - w_lse[~empty]) - tol_lse[~empty]
    assert bad.max(initial=0) <= 0, f"lse beyond by {bad.max()}"
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D, page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (256, 256), (256, 16)])
@pytest.mark.parametrize("heads, kv", [(1, 1), (4, 4), (8, 2), (5, 1), (16, 1), (6, 2), (8, 1)])
def test_decode(rmsq_gpu, dtype, D, page, heads, kv):
    """One query per request: one key, around tile and page ends, longer ones."""
    seq = [1, 15, 16, 17, 127, 128, 129, 300]
    check(rmsq_gpu, make([1] * len(seq), seq, heads, kv, D, page, dtype, seed=D + heads))


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D, heads, kv, page", [(64, 8, 1, 16), (128, 8, 2, 64), (128, 3, 1, 16), (256, 4, 2, 32)])
@pytest.mark.parametrize("window", [0, 1, 16, 100])
def test_several_queries(rmsq_gpu, dtype, D, heads, kv, page, window, variant):
    """Speculative tokens and prompts of odd lengths, with and without a
    window; a request without queries, one that is nothing but queries."""
    c = make([4, 1, 0, 33, 130], [77, 300, 20, 33, 391], heads, kv, D, page, dtype, seed=window)
    check(rmsq_gpu, c, window=window, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads, kv, page, q_lens, seq", [
    (1, 1, 16, [65], [65]),                        # one row more than the split kernel takes; a half tile
    (1, 1, 64, [128, 129], [128, 300]),
    (2, 2, 32, [257], [400]),                      # a tile and one row
    (8, 1, 16, [150, 1, 40], [150, 201, 127]),     # prompts and a decode in one batch
    (5, 1, 128, [60], [61]),                       # a group that does not divide the tile
    (16, 1, 16, [33, 9], [256, 129]),
    (6, 2, 256, [100, 90], [612, 90]),
])
def test_prompt(rmsq_gpu, dtype, D, heads, kv, page, q_lens, seq, variant):
    check(rmsq_gpu, make(q_lens, seq, heads, kv, D, page, dtype, seed=5 + D), variant=variant)
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 50, 128, 300])
def test_prompt_with_a_window(rmsq_gpu, D, window, variant):
    check(rmsq_gpu, make([200, 70], [700, 70], 4, 2, D, 16, "bf16", seed=window), window=window, variant=variant)


def test_prompts_of_the_automatic_choice(rmsq_gpu):
    """Enough rows for the prompt kernel to be chosen, a decode beside them."""
    check(rmsq_gpu, make([700, 1, 300], [700, 900, 420], 32, 2, 64, 16, "bf16", seed=70))
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_bad_pages_empty_rows_padding(rmsq_gpu, D, variant):
    """More queries than keys, pages outside the cache, garbage behind the
    last key, rows of padding, extreme and flat queries."""
    c = make([100, 80, 90], [60, 300, 0], 4, 2, D, 16, "bf16", seed=31, extra_rows=70)
    c["table"][1, 2], c["table"][1, 7], c["table"][1, 18] = -1, len(c["cache"]), -(2**31)
    codes, scales = ref.tiles(c["cache"], 16, D)
    codes[c["table"][0, 3], :, :, 12:] = 0xff
    scales[c["table"][0, 3], :, :, 12:] = 0xff
    c["q"][130:140] = 0
    c["q"][140:150] *= 1e3
    c["q64"] = c["q"].double().numpy()
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:2], 5.0, device="cuda")
    check(rmsq_gpu, c, out=out, lse=lse, variant=variant)
    assert (out[270:] == 3).all() and (lse[270:] == 5).all()


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_a_single_padded_request(rmsq_gpu, rows, variant):
    """A token buffer of 300 of which a single request fills some."""
    check(rmsq_gpu, make([rows], [rows + 33], 2, 1, 64, 16, "fp16", extra_rows=300 - rows), variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
def test_prompt_rising_logits(rmsq_gpu, variant):
    """The running maximum moves at every step, and differently per row."""
    c = make([300], [1000], 4, 1, 64, 16, "fp16", seed=3)
    codes, scales = ref.tiles(c["cache"], 16, 64)
    codes[:, 0] = 0x22
    for j in range(1000):
        scales[c["table"][0, j // 16], 0, :, j % 16] = 0x10 + j // 10
    c["q"], c["q64"] = ref.act(c["q64"] + np.linspace(-1, 1, 300)[:, None, None], torch.float16)
    check(rmsq_gpu, c, scale=0.5, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
def test_prompt_infinite_and_nan_queries_stay_in_their_rows(rmsq_gpu, variant):
    c = make([100, 30], [150, 30], 4, 1, 128, 16, "bf16", seed=6)
    good, good_lse = run(rmsq_gpu, c, variant=variant)
    q = c["q"].clone()
    q[10, 2, 5], q[99, 0, 0] = float("inf"), float("nan")
    out, lse = run(rmsq_gpu, c, q=q.cuda(), variant=variant)
    hit = torch.zeros(130, 4, dtype=torch.bool)
    hit[10, 2] = hit[99, 0] = True
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])
    assert torch.isnan(out[99, 0]).all()


@pytest.mark.parametrize("variant", VARIANTS)
def test_prompts_repeat_bit_for_bit_and_in_graphs(rmsq_gpu, variant):
    rq = rmsq_gpu
    c = make([500, 3, 260], [900, 1000, 260], 8, 2, 128, 64, "bf16", seed=40)
    a = run(rq, c, variant=variant)
    for _ in range(3):
        b = run(rq, c, variant=variant)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q, cache, table, seq = c["q"].cuda(), dev(c["cache"]), dev(c["table"]), dev(np.array(c["seq"], np.int32))
    start = torch.tensor([0, 500, 503, 763], dtype=torch.int32, device="cuda")
    g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
    ws = torch.empty(rq.paged_attention_workspace_bytes(763, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(763, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.paged_attention_nvfp4(q, cache, table, start, seq, g1, g2, 64, out=out, lse=lse, workspace=ws,
                                 variant=variant)
    graph.replay()
    assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    start.copy_(torch.tensor([0, 10, 700, 763]))        # other lengths, the same graph
    graph.replay()
    want = rq.paged_attention_nvfp4(q, cache, table, start, seq, g1, g2, 64, return_lse=True, variant=variant)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and rq.take_fault_flags() == 0


def test_rows_without_keys(rmsq_gpu):
    """Empty requests and more queries than keys: zeros and -inf."""
    c = make([1, 3, 5, 1], [0, 2, 0, 40], 8, 2, 128, 16, "bf16")
    out, lse = check(rmsq_gpu, c)
    assert torch.isinf(lse[0]).all() and torch.isinf(lse[1]).all() and torch.isfinite(lse[2]).all()


def test_bad_pages_are_left_out(rmsq_gpu):
    """Negative and too large page numbers, at ends and in the middle."""
    c = make([1, 1, 2], [200, 90, 130], 8, 2, 128, 16, "bf16", seed=2)
    c["table"][0, 3], c["table"][0, 12], c["table"][1, 0] = -1, len(c["cache"]), 2**31 - 1
    c["table"][2, :] = -5                      # a request with no page at all
    out, lse = check(rmsq_gpu, c)
    assert torch.isinf(lse[2:]).all()


def test_garbage_behind_the_last_key(rmsq_gpu):
    """Unwritten slots of the last page and spare pages hold 0xff (NaN scales)."""
    c = make([1, 2], [37, 130], 8, 2, 128, 64, "bf16", seed=4)
    clean = [t.clone() for t in run(rmsq_gpu, c)]
    codes, scales = ref.tiles(c["cache"], 64, 128)
    for r, n in enumerate(c["seq"]):
        last = c["table"][r, (n - 1) // 64]
        codes[last, :, :, (n - 1) % 64 + 1:] = 0xff
        scales[last, :, :, (n - 1) % 64 + 1:] = 0xff
    for a, b in zip(clean, run(rmsq_gpu, c)):
        assert torch.equal(a, b)


def test_rows_behind_the_last_request_stay(rmsq_gpu):
    c = make([1, 2, 1], [30, 40, 50], 8, 4, 64, 16, "fp16", extra_rows=9)
    out = torch.full((13, 8, 64), 3.0, dtype=torch.float16, device="cuda")
    lse = torch.full((13, 8), 5.0, device="cuda")
    check(rmsq_gpu, c, out=out, lse=lse)
    assert (out[4:] == 3).all() and (lse[4:] == 5).all()


@pytest.mark.parametrize("dtype, big", [("bf16", 1e30), ("bf16", 1e-30), ("fp16", 6e4), ("fp16", 6e-8)])
def test_extreme_queries(rmsq_gpu, dtype, big):
    """Query magnitudes at the ends of their type, one row unlike the next;
    the softmax scale keeps the logits ordinary."""
    c = make([1, 1, 1], [50, 260, 33], 4, 2, 64, 16, dtype, seed=8)
    x = np.random.default_rng(1).normal(0, 1, (3, 4, 64)) * big / 4
    c["q"], c["q64"] = ref.act(x, DT[dtype])
    check(rmsq_gpu, c, scale=float(np.float32(0.1 / big)) if big > 1 else min(0.1 / big, 1e20))


def test_infinite_and_nan_queries_stay_in_their_rows(rmsq_gpu):
    c = make([1, 1, 1, 1], [50, 60, 70, 80], 4, 1, 128, 16, "bf16", seed=6)
    good, good_lse = run(rmsq_gpu, c)
    q = c["q"].clone()
    q[1, 2, 5], q[2, 0, 0] = float("inf"), float("nan")
    out, lse = run(rmsq_gpu, c, q=q.cuda())
    hit = torch.zeros(4, 4, dtype=torch.bool)
    hit[1, 2] = hit[2, 0] = True
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])
    assert torch.isnan(out[1, 2]).any() and torch.isnan(out[2, 0]).all()


@pytest.mark.parametrize("sigma", [0.0, 30.0])
def test_flat_and_peaked_weights(rmsq_gpu, sigma):
    check(rmsq_gpu, make([1, 2, 1], [500, 130, 1], 8, 2, 128, 16, "bf16", sigma=sigma, seed=9))


def test_rising_logits_move_the_maximum(rmsq_gpu):
    """Keys that grow along the sequence: the running maximum moves at every step."""
    c = make([1], [1000], 4, 1, 64, 16, "fp16", seed=3)
    codes, scales = ref.tiles(c["cache"], 16, 64)
    codes[:, 0] = 0x22                                    # every element 1.0
    for j in range(1000):
        scales[c["table"][0, j // 16], 0, :, j % 16] = 0x10 + j // 10
    c["q"], c["q64"] = ref.act(np.abs(c["q64"]) + 0.5, torch.float16)
    check(rmsq_gpu, c, scale=0.5)


def test_a_long_sequence_split_over_the_card(rmsq_gpu):
    """One head over 20000 keys next to short ones; only a few rows are
    compared with float64, all of them with a second run bit for bit."""
    c = make([1, 1, 2], [20000, 3, 700], 4, 2, 128, 128, "bf16", seed=11)
    a = check(rmsq_gpu, c)
    b = run(rmsq_gpu, c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_strided_queries_shared_pages_and_reused_workspace(rmsq_gpu):
    """q as a column range of a qkv buffer; two requests on the same pages; a
    workspace full of NaN."""
    rq = rmsq_gpu
    c = make([1, 1], [90, 90], 8, 2, 128, 16, "bf16", seed=12)
    c["table"][1] = c["table"][0]
    wide = torch.randn(2, 12 * 128).bfloat16()
    wide[:, :1024] = c["q"].flatten(1)
    ws = torch.full((rq.paged_attention_workspace_bytes(2, 2, 8, 2, 128),), 0xff, dtype=torch.uint8, device="cuda")
    check(rq, c, q=wide.cuda()[:, :1024].unflatten(1, (8, 128)), workspace=ws)


def test_lengths_outside_the_buffers_are_clamped(rmsq_gpu):
    """Device-side lengths and offsets beyond the table, the tokens or below
    zero read nothing outside."""
    rq = rmsq_gpu
    c = make([1, 1, 1], [40, 40, 40], 4, 2, 64, 16, "bf16")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    one = torch.ones(1, device="cuda")
    for start, seq in (([0, 1, 2, 3], [2**31 - 1, -5, 40]), ([-9, 1, 2**31 - 1, 5], [40, 40, 40]), ([3, 2, 1, 0], [40] * 3)):
        out = rq.paged_attention_nvfp4(c["q"].cuda(), dev(c["cache"]), dev(c["table"]), dev(np.array(start, np.int32)),
                                       dev(np.array(seq, np.int32)), one, one, 16, out=torch.zeros_like(c["q"]).cuda())
        torch.cuda.synchronize()
        assert out.shape == (3, 4, 64)
    c = make([100, 100], [300, 300], 4, 2, 64, 16, "bf16")
    for start, seq in (([0, 100, 200], [2**31 - 1, -5]), ([-9, 2**31 - 1, 150], [300, 300]), ([200, 100, 0], [300, 1])):
        rq.paged_attention_nvfp4(c["q"].cuda(), dev(c["cache"]), dev(c["table"]), dev(np.array(start, np.int32)),
                                 dev(np.array(seq, np.int32)), one, one, 16, out=torch.zeros_like(c["q"]).cuda(),
                                 variant="pipelined")
        torch.cuda.synchronize()
    assert rq.take_fault_flags() == 0


def test_most_requests(rmsq_gpu):
    """As many requests as there may be, one key each: out is that value."""
    rq = rmsq_gpu
    R, page = rq.MAX_REQUESTS, 16
    cache = torch.zeros(rq.kv_cache_shape(R // 16, 1, 64, page), dtype=torch.uint8, device="cuda")
    k = torch.randn(R, 1, 64, device="cuda").bfloat16()
    slots = torch.arange(R, device="cuda")
    gs = torch.tensor([336.0], device="cuda")
    rq.kv_cache_store_nvfp4(k, k, slots, gs, gs, cache, page)
    _, v = rq.kv_cache_load_nvfp4(cache, slots, gs, gs, 64, page)
    # request r sees exactly slot r: window 1 at position r % 16 of page r / 16
    table = (torch.arange(R, device="cuda") // 16).int()[:, None].contiguous()
    seq = (torch.arange(R, device="cuda") % 16 + 1).int()
    start = torch.arange(R + 1, device="cuda").int()
    out = rq.paged_attention_nvfp4(k, cache, table, start, seq, gs, gs, page, window=1)
    assert torch.equal(out, v)


def test_graph_replay_follows_the_device_lengths(rmsq_gpu):
    rq = rmsq_gpu
    c = make([1, 1, 1], [30, 200, 64], 8, 2, 128, 16, "bf16", seed=21)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q, cache, table = c["q"].cuda(), dev(c["cache"]), dev(c["table"])
    start, seq = torch.arange(4, dtype=torch.int32, device="cuda"), dev(np.array(c["seq"], np.int32))
    g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
    ws = torch.empty(rq.paged_attention_workspace_bytes(3, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")

    def call():
        rq.paged_attention_nvfp4(q, cache, table, start, seq, g1, g2, 16, out=out, lse=lse, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1, 1, 1], [17, 208, 3], [30, 200, 64]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        q.neg_()
        graph.replay()
        got = out.clone(), lse.clone()
        call()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_a_decode_loop_of_the_operators_together(rmsq_gpu):
    """Slot map, QK-norm + RoPE, store, attention over a prompt step and three
    decode steps, against float64 attention over what the cache holds."""
    rq = rmsq_gpu
    import rmsq_inputs as ri
    R, nq, nkv, D, page, width, cap = 3, 8, 2, 128, 16, 6, 16
    torch.manual_seed(0)
    ctx = torch.zeros(R, dtype=torch.int32, device="cuda")
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(cap, device="cuda").int()
    left = torch.tensor([cap], dtype=torch.int32, device="cuda")
    cos_sin = torch.from_numpy(ri.rope_table(256, D)).cuda()
    w = (1 + 0.1 * torch.randn(D)).bfloat16().cuda()
    cache = torch.full(rq.kv_cache_shape(cap, nkv, D, page), 0xff, dtype=torch.uint8, device="cuda")
    gs = torch.tensor([2688 / 12.0], device="cuda")
    seq_host = [0] * R
    for q_lens in ([20, 1, 37], [1, 1, 1], [1, 1, 1], [2, 1, 0]):
        n = sum(q_lens)
        tokens = n + 2                                     # padded, as a captured step would be
        slots, pos, start, seq, left, status = rq.build_slot_map(
            ctx, torch.tensor(q_lens, dtype=torch.int32, device="cuda"), table, free, left, page, tokens)
        assert status.item() == 0
        qkv = torch.randn(tokens, (nq + 2 * nkv) * D, device="cuda").bfloat16()
        rq.qk_norm_rope(qkv, pos, cos_sin, w, w, 1e-6, nq, nkv, D)
        heads = qkv.unflatten(1, (nq + 2 * nkv, D))
        rq.kv_cache_store_nvfp4(heads[:, nq: nq + nkv], heads[:, nq + nkv:], slots, gs, gs, cache, page)
        out, lse = rq.paged_attention_nvfp4(heads[:, :nq], cache, table, start, seq, gs, gs, page, return_lse=True)
        seq_host = [a + b for a, b in zip(seq_host, q_lens)]
        assert seq.tolist() == seq_host
        q64 = heads[:n, :nq].double().cpu().numpy()
        w_out, w_lse, tol, tol_lse = ref.attention(q64, cache.cpu().numpy(), table.cpu().numpy(), q_lens, seq_host,
                                                   float(gs.item()), float(gs.item()), page, D ** -0.5, 0,
                                                   torch.finfo(torch.bfloat16).eps)
        assert (np.abs(out[:n].double().cpu().numpy() - w_out) <= tol).all()
        assert (np.abs(lse[:n].double().cpu().numpy() - w_lse) <= tol_lse).all()
        ctx = seq


def test_a_workspace_of_its_own_on_another_stream(rmsq_gpu):
    """Without a given workspace a call on a side stream keeps its own until
    that stream is done, whatever the current stream allocates meanwhile."""
    c = make([1] * 16, [2000] * 16, 32, 8, 128, 16, "bf16", seed=50)
    want = run(rmsq_gpu, c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append(run(rmsq_gpu, c, stream=s))
        torch.full((30 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_cpu_tensors_are_refused(rmsq_gpu):
    c = make([1], [20], 4, 2, 64, 16, "bf16")
    with pytest.raises(ValueError):
        run(rmsq_gpu, c, q=c["q"])


def test_an_attention_block_from_norm_to_output_projection(rmsq_gpu):
    """The operators as a decoder layer uses them, two steps captured in one
    graph and replayed: norm + quant, FP8 projection, QK-norm + RoPE, store,
    attention, quant, FP8 projection.  The graph's results are those of the
    calls made one by one, and each attention that of float64 over its cache."""
    rq = rmsq_gpu
    import rmsq_inputs as ri
    R, nq, nkv, D, H, page, cap = 4, 8, 2, 64, 512, 16, 40
    torch.manual_seed(2)
    E4M3 = torch.float8_e4m3fn
    w_qkv, w_o = (torch.randn(*s, device="cuda").to(E4M3) for s in (((nq + 2 * nkv) * D, H), (H, nq * D)))
    s_qkv, s_o = torch.rand(6, 4, device="cuda") * 0.05, torch.rand(4, 4, device="cuda") * 0.05
    cos_sin = torch.from_numpy(ri.rope_table(256, D)).cuda()
    wn, wh = torch.ones(H, device="cuda").bfloat16(), torch.ones(D, device="cuda").bfloat16()
    gs = torch.tensor([2688 / 8.0], device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    steps = [i32([30, 5, 1, 17]), i32([1, 1, 1, 1])]
    tokens = [60, 6]                                       # buffers, with padding rows
    xs = [torch.randn(t, H, device="cuda").bfloat16() for t in tokens]
    free, first_left = torch.randperm(cap, device="cuda").int(), i32([cap])
    ws = torch.empty(rq.paged_attention_workspace_bytes(60, R, nq, nkv, D), dtype=torch.uint8, device="cuda")

    def layer(table, cache):
        outs, ctx, left = [], i32_zero.clone(), first_left
        for new, n, x in zip(steps, tokens, xs):
            slots, pos, start, seq, left, status = rq.build_slot_map(ctx, new, table, free, left, page, n)
            q8, s8, r = rq.fused_add_rmsnorm_quant(x, x, wn, 1e-6, "fp8_group128_col+tma")
            qkv = rq.fp8_block_matmul(q8, s8, "fp8_group128_col+tma", w_qkv, s_qkv)
            rq.qk_norm_rope(qkv, pos, cos_sin, wh, wh, 1e-6, nq, nkv, D)
            heads = qkv.unflatten(1, (nq + 2 * nkv, D))
            rq.kv_cache_store_nvfp4(heads[:, nq: nq + nkv], heads[:, nq + nkv:], slots, gs, gs, cache, page)
            o = torch.zeros(n, nq, D, device="cuda", dtype=torch.bfloat16)
            rq.paged_attention_nvfp4(heads[:, :nq], cache, table, start, seq, gs, gs, page, out=o, workspace=ws)
            o8, so = rq.quant(o.flatten(1), "fp8_group128_row")
            y = rq.fp8_block_matmul(o8, so, "fp8_group128_row", w_o, s_o)
            outs.append((heads, o, y, status, seq, table.clone(), cache.clone()))
            ctx = seq
        return outs

    i32_zero = i32([0] * R)
    new_table = lambda: torch.full((R, 8), -1, dtype=torch.int32, device="cuda")  # noqa: E731
    new_cache = lambda: torch.zeros(rq.kv_cache_shape(cap, nkv, D, page), dtype=torch.uint8, device="cuda")  # noqa: E731
    plain = layer(new_table(), new_cache())
    table, cache = new_table(), new_cache()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed = layer(table, cache)
    for _ in range(2):
        table.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        for a, b, new in zip(plain, graphed, steps):
            n = int(new.sum())
            assert b[3].item() == 0 and torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])
            assert torch.equal(a[1][:n], b[1][:n]) and torch.equal(a[2][:n], b[2][:n])
    for (heads, o, y, _, seq, table, cache), new in zip(plain, steps):
        n = int(new.sum())
        w_out, _, tol, _ = ref.attention(heads[:n, :nq].double().cpu().numpy(), cache.cpu().numpy(), table.cpu().numpy(),
                                         new.tolist(), seq.tolist(), gs.item(), gs.item(), page, D ** -0.5, 0,
                                         torch.finfo(torch.bfloat16).eps)
        assert (np.abs(o[:n].double().cpu().numpy() - w_out) <= tol).all()
    assert rq.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
def test_many_short_requests_of_many_heads(rmsq_gpu, variant):
    """A thousand requests of 0 to 4 queries, 32 heads on one: rows on both
    sides of the prompt kernel's limit, lengths around a page."""
    rng = np.random.default_rng(60)
    q_lens = [int(x) for x in rng.integers(0, 5, 1000)]
    seq = [q + int(x) for q, x in zip(q_lens, rng.integers(0, 20, 1000))]
    check(rmsq_gpu, make(q_lens, seq, 32, 1, 64, 16, "bf16", seed=61), variant=variant)
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
def test_one_query_of_128_heads(rmsq_gpu, variant):
    check(rmsq_gpu, make([1, 1], [700, 129], 128, 1, 128, 64, "fp16", seed=62), variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_lens, seq", [([1, 1, 1], [40, 1, 5000]), ([30, 1, 20], [30, 200, 900])])
def test_a_nan_in_a_query_head_stays_there(rmsq_gpu, dtype, q_lens, seq, variant):
    """NaN in out and lse of that query head, alone or joined from parts; the
    others get what they get without it; a query without keys stays empty."""
    c = make(q_lens, seq, 8, 2, 128, 16, dtype, seed=63)
    want, want_lse = check(rmsq_gpu, c, variant=variant)
    hit = [(0, 3), (sum(q_lens) - 1, 0), (q_lens[0], 7)]
    for t, h in hit:
        c["q"][t, h, 77] = float("nan")
    out, lse = run(rmsq_gpu, c, variant=variant)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    for t, h in hit:
        bad[t, h] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    c["seq"] = [0] * len(seq)
    out, lse = run(rmsq_gpu, c, variant=variant)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_query_starts_that_do_not_ascend(rmsq_gpu):
    """Nothing outside the buffers is read or written, and requests in order
    keep their results."""
    rq = rmsq_gpu
    c = make([100, 50, 30], [200, 90, 30], 8, 1, 64, 16, "bf16", seed=64)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    gs = torch.tensor([c["k_gs"]], device="cuda")
    around = torch.full((3, 180, 8, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    for variant in VARIANTS:
        for starts in ([0, 180, 0, 180], [-5, 100, 90, 1000], [180, 0, 180, 0], [0, 2**31 - 1, -2**31, 50]):
            rq.paged_attention_nvfp4(c["q"].cuda(), dev(c["cache"]), dev(c["table"]), dev(np.array(starts, np.int64).astype(np.int32)),
                                     dev(np.array(c["seq"], np.int32)), gs, gs, 16, out=around[1], variant=variant)
            torch.cuda.synchronize()
    assert (around[0] == 7).all() and (around[2] == 7).all() and around[1].isfinite().all()
    assert rq.take_fault_flags() == 0


def make_exact_logits(dtype, D, q_lens, seq, *, order, seed):
    """Keys that are c_j in every dimension and queries that are +-2^i in every
    one, i spread over the type's range: every product and every partial sum
    has at most 6 + log2(D) bits, so the logits are exact in fp32 and lie from
    below 1 to 2^35 (fp16) or 2^120 (bf16) in units of log2.  c_j takes steps of at
    least 1/15, ascending, descending or mixed along the sequence."""
    c = make(q_lens, seq, 4, 2, D, 16, dtype, seed=seed)
    c["k_gs"] = np.float32(1.0)
    codes, scales = ref.tiles(c["cache"], 16, D)
    codes[:, 0] = 0x22                                    # every element 1.0
    steps = np.arange(0x18, 0x7f)                         # 2^-4 .. 448, eight steps an octave
    rng = np.random.default_rng(seed)
    for r, n in enumerate(seq):
        pick = np.sort(rng.integers(0, len(steps), n))
        pick = {"up": pick, "down": pick[::-1], "mixed": rng.permutation(pick)}[order]
        for j in range(n):
            scales[c["table"][r, j // 16], 0, :, j % 16] = steps[pick[j]]
    top = {"fp16": 15, "bf16": 100}[dtype]
    T = sum(q_lens)
    i = np.rint(np.linspace(-8, top, T * 4)).reshape(T, 4, 1)
    sign = np.where(rng.integers(0, 2, (T, 4, 1)) == 0, -1.0, 1.0)
    c["q"], c["q64"] = ref.act(np.broadcast_to(sign * 2.0 ** i, (T, 4, D)), DT[dtype])
    return c


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype, D", [("fp16", 64), ("fp16", 128), ("bf16", 64), ("bf16", 128), ("fp16", 256)])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("q_lens, seq", [([1] * 24, [300 + 16 * r for r in range(24)]), ([130, 70], [130, 900]),
                                         ([3], [9000])])
def test_large_logits(rmsq_gpu, dtype, D, order, q_lens, seq, variant):
    """Finite inputs whose logits are far beyond 2^24: the largest one's weight
    is 1, whatever their magnitude, and lse is finite.

    The logits are exact here, so that beside the roundings of
    tests/_serve_ref.py (output, f16 weights, sums) there are: the factor that
    turns logits into powers of two, off by three roundings (2^-22 relative),
    which changes a weight e^-g by g e^-g 2^-22 < 2^-23; the subtraction of the
    maximum, which for maxima up to 2^10 may round by 2^-14 and again where the
    maximum has moved since (2 ln2 2^-14 < 2^-13), and the exponential (2^-21).
    lse: its own roundings (2^-22 relative), 2^-13 and the sums."""
    c = make_exact_logits(dtype, D, q_lens, seq, order=order, seed=D)
    out, lse = run(rmsq_gpu, c, variant=variant)
    eps = torch.finfo(DT[dtype]).eps
    w_out, w_lse, _, _ = ref.attention(c["q64"], c["cache"], c["table"], q_lens, seq, 1.0, float(c["v_gs"]), 16, D ** -0.5,
                                       0, eps)
    most = max(np.abs(ref.values(*ref.tiles(c["cache"], 16, D), float(c["v_gs"]))[:, 1]).max(), 0.0)
    n = max(seq)
    tol = eps / 2 * np.abs(w_out) + most * (2.0 ** -11 + 2.0 ** -12 + 2 * n * 2.0 ** -23 + n * 2.0 ** -34)
    tol_lse = 2.0 ** -21 * np.abs(w_lse) + 2.0 ** -12 + n * 2.0 ** -23
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all() and np.isfinite(s).all()
    assert (np.abs(o - w_out) <= tol).all(), np.abs(o - w_out).max()
    assert (np.abs(s - w_lse) <= tol_lse).all(), (np.abs(s - w_lse) / tol_lse).max()
    assert (np.abs(w_lse) > 2.0 ** 13).any()
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype, q", [("fp16", 6e4), ("fp16", -6e4), ("bf16", 1e20), ("bf16", -1e38)])
@pytest.mark.parametrize("rows", [1, 9, 90])
def test_one_dominant_key(rmsq_gpu, dtype, q, rows, variant):
    """Every element of the dominant key at its largest and the others at
    random: out is that key's value, off by its own rounding and the weight's
    (which is 2^9 exactly) alone; lse its logit (bf16 queries of 1e38: beyond
    fp32, +inf)."""
    c = make([rows], [400], 8, 1, 128, 16, dtype, seed=65)
    c["k_gs"] = np.float32(2.0)
    codes, scales = ref.tiles(c["cache"], 16, 128)
    codes[c["table"][0, 7], 0, :, 5], scales[c["table"][0, 7], 0, :, 5] = 0x77 if q > 0 else 0xff, 0x7e   # key 117
    c["q"], c["q64"] = ref.act(np.full((rows, 8, 128), q), DT[dtype])
    out, lse = run(rmsq_gpu, c, variant=variant)
    eps = torch.finfo(DT[dtype]).eps
    w_out, w_lse, _, _ = ref.attention(c["q64"], c["cache"], c["table"], [rows], [400], 2.0, float(c["v_gs"]), 16,
                                       128 ** -0.5, 0, eps)
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - w_out) <= np.abs(w_out) * (eps / 2 + 2.0 ** -21)).all(), np.abs(o - w_out).max()
    if abs(q) < 1e30:
        assert (np.abs(s - w_lse) <= np.abs(w_lse) * (130 + 8) * 2.0 ** -23).all()
    else:
        assert (s == np.inf).all()


def launches(rq, c, **kw):
    """Kernels that a call launches: the nodes of its graph."""
    import ctypes
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    start = np.concatenate([[0], np.cumsum(c["q_lens"])]).astype(np.int32)
    one = torch.ones(1, device="cuda")
    args = [c["q"].cuda(), dev(c["cache"]), dev(c["table"]), dev(start), dev(np.array(c["seq"], np.int32)), one, one, c["page"]]
    rq.paged_attention_nvfp4(*args, **kw)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        rq.paged_attention_nvfp4(*args, **kw)
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcudart.so.13").cudaGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None,
                                                            ctypes.byref(n)) == 0
    return n.value


def test_the_automatic_choice_launches_what_the_step_needs(rmsq_gpu):
    """A large decode batch has no use for the kernel of prompts (beside the
    split and its join); with a bound on the queries neither has a batch of
    speculative tokens."""
    def count(q_lens, seq, **kw):
        return launches(rmsq_gpu, make(q_lens, seq, 32, 8, 64, 16, "bf16", seed=70), **kw)

    assert count([1] * 300, [40] * 300) == 2
    assert count([1] * 290 + [0] * 10, [40] * 300) == 2
    assert count([4] * 100, [40] * 100, max_query=4) == 2
    assert count([1] * 40 + [400], [40] * 40 + [400]) == 3
    assert count([1] * 40 + [400], [40] * 40 + [400], max_query=400) == 3
    assert count([400], [400]) == 1


@pytest.mark.parametrize("max_query", [1, 30, 400, 10**9])
@pytest.mark.parametrize("q_lens, seq", [([1] * 40, [60] * 40), ([1, 400, 30], [50, 450, 30]), ([300], [300])])
def test_a_bound_on_the_queries_changes_no_result(rmsq_gpu, q_lens, seq, max_query):
    """Right, too high and too low."""
    for variant in ("auto", "pipelined"):
        check(rmsq_gpu, make(q_lens, seq, 8, 2, 64, 16, "bf16", seed=71), max_query=max_query, variant=variant)
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads, kv", [(8, 1), (8, 8), (16, 1), (32, 2), (12, 1)])
def test_decodes_beside_a_prompt(rmsq_gpu, dtype, D, heads, kv):
    """One batch for both kernels: groups on both sides of a row block, a few
    requests of several queries among the decodes, lengths around a tile."""
    q_lens = [1] * 20 + [300] + [1, 3, 0, 4, 1, 60] + [1] * 5
    seq = [10 * i + 1 for i in range(20)] + [420] + [128, 3, 50, 129, 500, 64] + [257, 1, 16, 300, 0]
    for variant in ("auto", "pipelined"):
        check(rmsq_gpu, make(q_lens, seq, heads, kv, D, 16, dtype, seed=72), variant=variant)
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens, seq", [
    ([1] * 12 + [40] + [300] + [1], [30] * 12 + [5000] + [300] + [700]),   # few rows on a long context beside a prompt
    ([20] * 24, [20 + 40 * i for i in range(24)]),                         # enough of them for the card, of all lengths
    ([0, 17, 300, 0, 90, 33, 16], [0, 2500, 300, 40, 1000, 20, 900]),      # on both sides of the rule, empty requests
    ([1] * 33 + [0, 20, 300, 17, 17, 17, 9], [i + 1 for i in range(33)] + [0, 1500, 310, 17, 140, 600, 3000]),  # more than 32
])
def test_requests_shared_out_between_the_kernels(rmsq_gpu, q_lens, seq, D, window):
    """Every request is exactly one kernel's, whatever the lengths beside it."""
    c = make(q_lens, seq, 32, 8, D, 16, "bf16", seed=73)
    assert launches(rmsq_gpu, c, window=window) == 3        # both kernels and the join
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    check(rmsq_gpu, c, window=window, out=out)
    assert rmsq_gpu.take_fault_flags() == 0


def test_few_rows_on_a_long_context_beside_decodes_stay_divided(rmsq_gpu):
    """The automatic choice takes no longer than twice the kernel that divides
    the keys (the other one walks them in a few CTAs: five times)."""
    rq = rmsq_gpu
    q_lens, seq, heads, kv, D, page = [1] * 128 + [9], [2000] * 128 + [100000], 64, 8, 128, 64
    pages = 1600
    table = torch.randint(0, pages, (129, 1563), device="cuda").int()
    cache = torch.randint(0, 0x40, rq.kv_cache_shape(pages, kv, D, page), device="cuda").to(torch.uint8)
    q = torch.randn(137, heads, D, device="cuda").bfloat16()
    start = torch.tensor([0] + q_lens, device="cuda").cumsum(0).int()
    seqs, one = torch.tensor(seq, device="cuda").int(), torch.ones(1, device="cuda")
    ws = torch.empty(rq.paged_attention_workspace_bytes(137, 129, heads, kv, D), dtype=torch.uint8, device="cuda")

    def us(variant):
        call = lambda: rq.paged_attention_nvfp4(q, cache, table, start, seqs, one, one, page, workspace=ws, variant=variant)  # noqa: E731
        call()
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                call()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 250)
        return min(times)

    assert us("auto") < 2 * us("direct")


def test_a_replayed_graph_follows_requests_that_change_hands(rmsq_gpu):
    """Lengths in device memory move requests from one kernel to the other
    between replays of one graph, with the workspace the call took itself."""
    rq = rmsq_gpu
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    c = make([340, 30, 30], [340, 2000, 60], 32, 8, 64, 16, "bf16", seed=74)
    assert launches(rq, c) == 3
    q, cache, table = c["q"].cuda(), dev(c["cache"]), dev(c["table"])
    # rows of every request on pages of the longest one
    table[:] = table[1]
    c["table"] = table.cpu().numpy()
    start, seq = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
    out, lse = torch.empty_like(q), torch.empty(400, 32, device="cuda")
    call = lambda: rq.paged_attention_nvfp4(q, cache, table, start, seq, g1, g2, 16, out=out, lse=lse)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for q_lens, lens in (([340, 30, 30], [340, 2000, 60]), ([20, 360, 20], [2000, 360, 20]), ([1, 1, 1], [7, 1999, 64]),
                         ([100, 100, 100], [1900, 100, 150]), ([0, 0, 400], [5, 0, 400])):
        start.copy_(torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32))
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        got, got_lse, n = out.clone(), lse.clone(), sum(q_lens)
        call()
        assert torch.equal(got, out) and torch.equal(got_lse[:n], lse[:n]) and (got[n:] == 3).all()
        w_out, w_lse, tol, tol_lse = ref.attention(c["q64"][:n], c["cache"], c["table"], q_lens, lens, float(c["k_gs"]),
                                                   float(c["v_gs"]), 16, 64 ** -0.5, 0, torch.finfo(torch.bfloat16).eps)
        assert (np.abs(got[:n].double().cpu().numpy() - w_out) <= tol).all()
    assert rq.take_fault_flags() == 0

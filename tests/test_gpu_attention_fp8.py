"""Attention over the paged FP8 cache on the GPU, against float64 with
tolerances derived beside the reference (tests/_serve8_ref.py)."""
import numpy as np
import pytest
import torch

import _serve8_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
VARIANTS = ("direct", "pipelined")


def make(q_lens, seq_lens, heads, kv, D, page, dtype, *, seed=0, extra_rows=0, sigma=1.0, spare=3, k_scale=(117, 123),
         v_scale=(110, 126)):
    """Codes of every value but NaN, scales over a range; what lies behind the last
    token of a request, and pages of nobody, hold NaN codes and any scale byte."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-s // page)) for s in seq_lens]
    pages, width = sum(need) + spare, max(need) + 1
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(seq_lens), width), -1, np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at: at + m]
        at += m
    codes = rng.integers(0, 256, (pages, 2, kv, page, D), dtype=np.uint8)
    codes[(codes & 127) == 127] = 3
    scales = np.stack([rng.integers(*s, (pages, kv, page // 16), dtype=np.uint8) for s in (k_scale, v_scale)], 1)
    used = np.zeros((pages, page), bool)
    for r, s in enumerate(seq_lens):
        j = np.arange(s)
        used[table[r, j // page], j % page] = True
    codes[~used[:, None, None].repeat(2, 1).repeat(kv, 2)] = rng.choice(np.array([0x7f, 0xff, 0x7e], np.uint8))
    blocks = used.reshape(pages, 1, 1, page // 16, 16).any(-1)
    scales[~np.broadcast_to(blocks, scales.shape)] = rng.choice(np.array([0, 255, 254], np.uint8))
    T = sum(q_lens) + extra_rows
    q = torch.from_numpy(rng.normal(0, sigma, (T, heads, D))).to(DT[dtype])
    return {"q": q, "q64": q.double().numpy(), "codes": codes, "scales": scales, "table": table, "q_lens": list(q_lens),
            "seq": list(seq_lens), "page": page, "D": D, "dtype": dtype}


def run(rq, c, *, window=0, scale=None, stream=None, **kw):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    start = np.concatenate([[0], np.cumsum(c["q_lens"])]).astype(np.int32)
    return rq.paged_attention_fp8(kw.pop("q", c["q"].cuda()), dev(c["codes"]), dev(c["scales"]), dev(c["table"]), dev(start),
                                  dev(np.array(c["seq"], np.int32)), scale, window=window, return_lse=True, stream=stream, **kw)


def check(rq, c, *, window=0, scale=None, **kw):
    n = sum(c["q_lens"])
    out, lse = run(rq, c, window=window, scale=scale, **kw)
    eps = torch.finfo(DT[c["dtype"]]).eps
    want, w_lse, tol, tol_lse = ref.attention(c["q64"][:n], c["codes"], c["scales"], c["table"], c["q_lens"], c["seq"],
                                              c["D"] ** -0.5 if scale is None else scale, window, eps)
    o, s = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    empty = np.isinf(w_lse)
    assert np.array_equal(np.isinf(s), empty) and (s[empty] < 0).all() and (o[empty] == 0).all()
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(o), bad), "NaN at other places"
    assert np.array_equal(np.isnan(s), np.isnan(w_lse))
    off = (np.abs(o - want) - tol)[~bad]
    assert off.max(initial=0) <= 0, f"out off by up to {np.nanmax(np.abs(o - want))}, {(off > 0).sum()} beyond"
    off = np.abs(s[~empty] - w_lse[~empty]) - tol_lse[~empty]
    assert np.nanmax(off, initial=0) <= 0, f"lse beyond by {np.nanmax(off)}"
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D, page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (256, 256), (256, 16)])
@pytest.mark.parametrize("heads, kv", [(1, 1), (4, 4), (8, 2), (5, 1), (16, 1), (6, 2), (40, 1)])
def test_decode(rmsq_gpu, dtype, D, page, heads, kv):
    """One query per request: one key, around block, tile and page ends, longer ones."""
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
    (1, 1, 16, [65], [65]),
    (1, 1, 64, [128, 129], [128, 300]),
    (2, 2, 32, [257], [400]),
    (8, 1, 16, [150, 1, 40], [150, 201, 127]),
    (5, 1, 128, [60], [61]),
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


@pytest.mark.parametrize("q_lens", [
    [76], [77], [300], [4000], [64, 1, 33, 0, 40], [20, 2, 90] * 11, [1] * 37 + [95], [1] * 40, [17] * 40 + [200]])
@pytest.mark.parametrize("D, heads, kv", [(64, 8, 4), (128, 4, 1)])
def test_prompts_in_tiles_and_pairs_of_tiles(rmsq_gpu, D, heads, kv, q_lens):
    """CTAs of 128 rows where they fit the card together, of 256 where not; up to 32 requests and more."""
    seq = [q + 11 * r % 170 for r, q in enumerate(q_lens)]
    check(rmsq_gpu, make(q_lens, seq, heads, kv, D, 32, "bf16", seed=len(q_lens)), variant="pipelined")


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_empty_rows_padding(rmsq_gpu, D, variant):
    """More queries than keys, pages outside the cache, rows of padding, extreme
    and flat queries."""
    c = make([100, 80, 90, 1], [60, 300, 0, 40], 4, 2, D, 16, "bf16", seed=31, extra_rows=70)
    c["table"][1, 2], c["table"][1, 7], c["table"][1, 18] = -1, len(c["codes"]), -(2**31)
    c["table"][3, 0] = c["table"][3, 1] = c["table"][3, 2] = -1         # nothing to see
    c["q"][130:140] = 0
    c["q"][140:150] *= 1e3
    c["q64"] = c["q"].double().numpy()
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:2], 5.0, device="cuda")
    check(rmsq_gpu, c, out=out, lse=lse, variant=variant)
    assert (out[271:] == 3).all() and (lse[271:] == 5).all()


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("k_scale, v_scale", [((88, 187), (88, 187)), ((100, 118), (140, 150)), ((119, 120), (88, 89)),
                                              ((119, 120), (186, 188))])
def test_scales_over_their_range(rmsq_gpu, k_scale, v_scale, variant):
    """Blocks of very different scale side by side: logits of any magnitude,
    value scales that rise and fall along the keys, and so far apart that the
    weights of the small ones vanish."""
    c = make([90, 2, 1], [400, 333, 150], 4, 1, 64, 16, "bf16", seed=k_scale[0] + v_scale[0], k_scale=k_scale, v_scale=v_scale)
    check(rmsq_gpu, c, variant=variant)
    assert rmsq_gpu.take_fault_flags() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 40])
def test_large_values_before_the_window(rmsq_gpu, D, window, variant):
    """Rows that see nothing of the first tiles, whose value scales are far above
    one, and rows that see nothing at all."""
    c = make([150, 70, 3], [290, 60, 200], 4, 2, D, 16, "bf16", seed=window, v_scale=(128, 187))
    check(rmsq_gpu, c, window=window, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("rising", [True, False])
def test_values_that_grow_along_the_keys(rmsq_gpu, rising, variant):
    """The value scale of a block 2^1 (2^-1) times the one before it, and equal
    keys: early queries see only the small ones, with their own precision."""
    c = make([200], [200], 2, 1, 128, 16, "fp16", seed=6, k_scale=(100, 101))
    order = np.arange(13) if rising else np.arange(13)[::-1]
    c["scales"][c["table"][0, :13], 1, 0, 0] = 108 + order
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
def test_rising_logits(rmsq_gpu, variant):
    """The running maximum moves at every step, and differently per row."""
    c = make([300], [1000], 4, 1, 64, 16, "fp16", seed=3)
    c["codes"][:, 0] = 0x38                                             # 1.0
    c["scales"][c["table"][0, :63], 0, 0, 0] = 110 + np.arange(63) // 4
    c["q"] = torch.rand(300, 4, 64, dtype=torch.float64).to(torch.float16)
    c["q64"] = c["q"].double().numpy()
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("window", [0, 40])
def test_nan_keys_reach_those_who_see_them(rmsq_gpu, window, variant):
    """A key with a NaN code amid a prompt: its queries and the later ones (within
    the window) give NaN, the earlier ones do not; NaN codes of values are 448."""
    c = make([150, 1, 70], [260, 90, 70], 4, 2, 64, 16, "bf16", seed=9)
    put = lambda r, j, side, head, code: c["codes"].__setitem__((c["table"][r, j // 16], side, head, j % 16, 5), code)  # noqa: E731
    put(0, 170, 0, 0, 0x7f)
    put(2, 33, 0, 1, 0xff)
    put(0, 3, 1, 1, 0x7f)
    put(1, 50, 1, 0, 0xff)
    check(rmsq_gpu, c, window=window, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_not_finite_queries_stay_their_own(rmsq_gpu, what, variant):
    c = make([90, 1], [200, 130], 4, 2, 64, 16, "bf16", seed=19)
    clean, _ = run(rmsq_gpu, c, variant=variant)
    q = c["q"].clone()
    q[17, 1, 3] = what
    out, lse = run(rmsq_gpu, c, q=q.cuda(), variant=variant)
    assert out[17, 1].isnan().all() and lse[17, 1].isnan()
    out[17, 1] = clean[17, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("scale", [1e-6, 3.0, 1e30])
def test_softmax_scales(rmsq_gpu, scale, variant):
    """From flat weights to a single key's (ties are decided by the exact logit)."""
    c = make([70, 1], [150, 99], 2, 1, 64, 16, "fp16", seed=23)
    out, lse = run(rmsq_gpu, c, scale=scale, variant=variant)
    if scale < 1e20:
        check(rmsq_gpu, c, scale=scale, variant=variant)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_strided_queries_and_outputs_given(rmsq_gpu):
    """q as a column range of a qkv buffer; a workspace and outputs of one's own;
    the codes as float8_e4m3fn."""
    c = make([1] * 9, [50 + 30 * i for i in range(9)], 8, 2, 128, 32, "bf16", seed=41)
    buf = torch.zeros(9, 12, 128, dtype=torch.bfloat16, device="cuda")
    buf[:, :8] = c["q"].cuda()
    ws = torch.empty(rmsq_gpu.paged_attention_workspace_bytes(9, 9, 8, 2, 128), dtype=torch.uint8, device="cuda")
    a, _ = check(rmsq_gpu, c, q=buf[:, :8], workspace=ws)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    b = rmsq_gpu.paged_attention_fp8(c["q"].cuda(), dev(c["codes"]).view(torch.float8_e4m3fn), dev(c["scales"]), dev(c["table"]),
                                     dev(np.arange(10, dtype=np.int32)), dev(np.array(c["seq"], np.int32)))
    assert torch.equal(a, b)


@pytest.mark.parametrize("D, heads, kv", [(64, 8, 8), (128, 32, 4), (256, 8, 2)])
def test_long_ragged_decode_and_determinism(rmsq_gpu, D, heads, kv):
    """Many requests cut over the whole card."""
    rng = np.random.default_rng(D)
    seq = [int(x) for x in rng.integers(1, 900, 20)] + [5000]
    c = make([1] * 21, seq, heads, kv, D, 64, "bf16", seed=D)
    a = check(rmsq_gpu, c)
    for _ in range(3):
        b = run(rmsq_gpu, c)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("requests", [30, 130, 500])
@pytest.mark.parametrize("D, heads, kv", [(64, 8, 8), (128, 12, 4), (256, 6, 2)])
def test_many_requests_of_one_to_three_tiles(rmsq_gpu, D, heads, kv, requests):
    """Fewer and more tiles of 128 keys than CTAs; requests without queries or keys among them."""
    rng = np.random.default_rng(requests + D)
    q_lens = rng.integers(0, 4, requests).tolist()
    seq = [0 if q == 0 and r % 2 else q + int(rng.integers(0, 380)) for r, q in enumerate(q_lens)]
    check(rmsq_gpu, make(q_lens, seq, heads, kv, D, 16, "bf16", seed=requests), variant="direct")


def test_no_tokens_no_requests_no_pages(rmsq_gpu):
    rq = rmsq_gpu
    c = make([1], [20], 2, 1, 64, 16, "bf16")
    empty = dict(c, q=c["q"][:0], q_lens=[0])
    out, _ = run(rq, empty)
    assert out.shape == (0, 2, 64)
    none = dict(c, codes=c["codes"][:0], scales=c["scales"][:0])
    out, lse = run(rq, none)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_offsets_beyond_32_bits(rmsq_gpu):
    """A cache of more than 4 GB; its last pages hold the request."""
    rq = rmsq_gpu
    kv, D, page = 8, 128, 256
    pages = (5 << 30) // (2 * kv * page * D)
    c = make([1], [1000], 16, kv, D, page, "bf16", seed=77, spare=0)
    cache = torch.full((pages, 2, kv, page, D), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, 2, kv, page // 16), 255, dtype=torch.uint8, device="cuda")
    n = len(c["codes"])
    cache[pages - n:] = torch.from_numpy(c["codes"]).cuda()
    scales[pages - n:] = torch.from_numpy(c["scales"]).cuda()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    table = np.where(c["table"] >= 0, c["table"] + pages - n, -1).astype(np.int32)
    args = [dev(table), dev(np.array([0, 1], np.int32)), dev(np.array([1000], np.int32))]
    want, _ = run(rq, c)
    assert torch.equal(rq.paged_attention_fp8(c["q"].cuda(), cache, scales, *args), want)


def test_a_replayed_graph_whose_requests_change(rmsq_gpu):
    """Captured once; replayed with other lengths, tables and prompts beside decodes."""
    rq = rmsq_gpu
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    steps = [make([1] * 6 + [100], [40, 300, 5, 900, 77, 130, 260], 8, 2, 64, 16, "bf16", seed=91),
             make([100] + [1] * 6, [100, 12, 500, 31, 64, 640, 17], 8, 2, 64, 16, "bf16", seed=92)]
    pages = max(len(c["codes"]) for c in steps)
    width = max(c["table"].shape[1] for c in steps)
    for c in steps:
        grow = lambda a: np.concatenate([a, np.zeros((pages - len(a),) + a.shape[1:], a.dtype)])  # noqa: E731
        c["codes"], c["scales"] = grow(c["codes"]), grow(c["scales"])
        c["table"] = np.pad(c["table"], ((0, 0), (0, width - c["table"].shape[1])), constant_values=-1)
        c["start"] = np.concatenate([[0], np.cumsum(c["q_lens"])]).astype(np.int32)
        c["seq_lens"] = np.array(c["seq"], np.int32)
    names = ("codes", "scales", "table", "start", "seq_lens")
    bufs = [dev(steps[0][k]) for k in names]
    q = steps[0]["q"].cuda()
    rq.paged_attention_fp8(q, *bufs, return_lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = rq.paged_attention_fp8(q, *bufs, return_lse=True)
    for c in (steps[1], steps[0], steps[1]):
        for b, k in zip(bufs, names):
            b.copy_(dev(c[k]))
        q.copy_(c["q"].cuda())
        graph.replay()
        torch.cuda.synchronize()
        want, w_lse = check(rq, c)
        assert torch.equal(out, want) and torch.equal(lse, w_lse)
    assert rq.take_fault_flags() == 0


def test_the_path_together(rmsq_gpu):
    """Slot map, rotation with three axes, store and attention as a step runs
    them, for three steps of four requests, against float64 on what the cache
    then holds."""
    rq = rmsq_gpu
    torch.manual_seed(3)
    nq, h, D, page, R = 8, 2, 128, 32, 4
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, scales = (torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(64, h, D, page))
    table = torch.full((R, 20), -1, dtype=torch.int32, device="cuda")
    free, left, ctx = torch.randperm(64, device="cuda").int(), i32([64]), i32([0] * R)
    angle = torch.arange(2000, dtype=torch.float64)[:, None] * 1e4 ** -(torch.arange(64, dtype=torch.float64) / 64)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    q_w, k_w = ((1 + 0.1 * torch.randn(D, device="cuda")).bfloat16() for _ in range(2))
    for new in ([200, 3, 0, 77], [1, 1, 50, 1], [1, 4, 1, 1]):
        T = 300
        slots, pos, start, seq, left, status = rq.build_slot_map(ctx, i32(new), table, free, left, page, T)
        assert status.item() == 0
        qkv = torch.randn(T, (nq + 2 * h) * D, device="cuda").bfloat16()
        pos3 = torch.stack([pos, torch.where(pos >= 0, pos // 7, pos), torch.where(pos >= 0, pos % 7, pos)])
        rq.qk_norm_mrope(qkv, pos3, cs, q_w, k_w, 1e-6, nq, h, D, (24, 20, 20), interleaved=True)
        heads = qkv.unflatten(1, (nq + 2 * h, D))
        rq.kv_cache_store_fp8(heads[:, nq: nq + h], heads[:, nq + h:], slots, cache, scales)
        out, lse = rq.paged_attention_fp8(heads[:, :nq], cache, scales, table, start, seq, return_lse=True)
        n = sum(new)
        want, w_lse, tol, tol_lse = ref.attention(heads[:n, :nq].double().cpu().numpy(), cache.cpu().numpy(),
                                                  scales.cpu().numpy(), table.cpu().numpy(), new, seq.tolist(), D ** -0.5, 0,
                                                  torch.finfo(torch.bfloat16).eps)
        assert (np.abs(out[:n].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse[:n].double().cpu().numpy() - w_lse) <= tol_lse).all()
        ctx = seq
    assert rq.take_fault_flags() == 0

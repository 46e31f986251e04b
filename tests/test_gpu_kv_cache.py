"""Slot maps and the paged NVFP4 cache's store and load on the GPU, against
plain references: integers and cache bytes have to be equal."""
import numpy as np
import pytest
import torch

import _serve_ref as ref
import oracle

pytestmark = pytest.mark.gpu


def _slots(rq, ctx, qlen, width, page, max_tokens, num_free, *, capacity=None, seed=0, holes=False):
    rng = np.random.default_rng(seed)
    R = len(ctx)
    capacity = num_free + 3 if capacity is None else capacity
    held = [min(width, max(0, -(-c // page))) for c in ctx]
    ids = rng.permutation(sum(held) + capacity + 5).astype(np.int32)
    table = np.full((R, width), -7, np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at: at + h]
        at += h
    if holes and R and held[0]:
        table[0, 0] = -1
    free = ids[at: at + capacity]
    want = ref.slot_map(ctx, qlen, table, free, num_free, page, max_tokens)
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    d_ctx, d_q, d_table, d_free, d_n = dev(ctx), dev(qlen), dev(table).reshape(R, width), dev(free), dev([num_free])
    keep = [t.clone() for t in (d_ctx, d_q, d_free, d_n)]
    got = rq.build_slot_map(d_ctx, d_q, d_table, d_free, d_n, page, max_tokens)
    torch.cuda.synchronize()
    for name, g, w in zip(("slots", "positions", "start", "seq", "free", "status"), got, want):
        assert g.flatten().tolist() == (list(w) if isinstance(w, list) else [w]), name
    assert np.array_equal(d_table.cpu().numpy(), want[6])
    for a, b in zip(keep, (d_ctx, d_q, d_free, d_n)):
        assert torch.equal(a, b)
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("ctx, qlen", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17], [1]), ([255], [1]), ([256], [2]),
    ([5, 0, 300, 31], [1, 33, 0, 700]),
    ([0] * 40, [0] * 39 + [1]),
    (list(range(0, 600, 1)), [1] * 600),
    ([(7 * i) % 900 for i in range(1500)], [(i * i) % 37 for i in range(1500)]),
])
def test_slot_map(rmsq_gpu, page, ctx, qlen):
    width = max(-(-(c + q) // page) for c, q in zip(ctx, qlen)) + 2
    need = sum(-(-(c + q) // page) - -(-c // page) for c, q in zip(ctx, qlen))
    for pad in (0, 5, 1200):
        _slots(rmsq_gpu, ctx, qlen, width, page, sum(qlen) + pad, need + pad % 3, seed=pad)
    if need == 0:
        _slots(rmsq_gpu, ctx, qlen, width, page, sum(qlen), 0, capacity=0)


def test_slot_map_most_requests_and_none(rmsq_gpu):
    R = rmsq_gpu.MAX_REQUESTS
    _slots(rmsq_gpu, [16 * (i % 5) for i in range(R)], [1 + (i % 3 == 0) for i in range(R)], 7, 16, 2 * R, 2 * R)
    _slots(rmsq_gpu, [], [], 3, 16, 4, 2)
    _slots(rmsq_gpu, [], [], 0, 16, 0, 0, capacity=0)


def test_slot_map_negative_page_gives_no_slot(rmsq_gpu):
    got = _slots(rmsq_gpu, [3, 40], [2, 9], 8, 16, 12, 4, holes=True)
    assert got[0][:2].tolist() == [-1, -1]


@pytest.mark.parametrize("ctx, qlen, width, max_tokens, num_free, capacity, bits", [
    ([30, 5], [40, 20], 9, 60, 2, 5, 1),       # four pages needed, two free
    ([30, 5], [40, 20], 3, 60, 9, 9, 2),       # five columns needed
    ([30, 5], [40, 20], 9, 59, 9, 9, 4),
    ([30, -5], [40, 20], 9, 60, 9, 9, 8),
    ([30, 5], [40, -1], 9, 60, 9, 9, 8),
    ([30, 5], [40, 20], 9, 60, -1, 9, 8),
    ([30, 5], [40, 20], 9, 60, 10, 9, 8),
    ([2**31 - 1, 5], [2**31 - 1, 20], 9, 60, 9, 9, 1 | 2 | 4),
])
def test_slot_map_reports_and_assigns_nothing(rmsq_gpu, ctx, qlen, width, max_tokens, num_free, capacity, bits):
    got = _slots(rmsq_gpu, ctx, qlen, width, 16, max_tokens, num_free, capacity=capacity)
    assert got[5].item() == bits


DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _kv(rng, n, h, D, dtype):
    x = rng.normal(0, 1, (n, h, D)) * np.exp2(rng.integers(-6, 5, (n, h, D // 16)).repeat(16, -1))
    x[rng.random((n, h, D // 16)).repeat(16, -1) < 0.03] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n, h, D, page", [(1, 1, 64, 16), (3, 2, 64, 32), (37, 4, 128, 16), (200, 1, 128, 256),
                                           (65, 8, 128, 64), (19, 3, 256, 128), (2500, 2, 256, 16)])
def test_store_and_load(rmsq_gpu, dtype, n, h, D, page):
    rq = rmsq_gpu
    rng = np.random.default_rng(n * 7 + D)
    k, v = _kv(rng, n, h, D, dtype), _kv(rng, n, h, D, dtype)
    gs = [np.float32(2688 / 97.3), np.float32(2688 / 211.7)]
    pages = -(-n // page) + 2
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 2:
        slots[1], slots[2] = -1, pages * page          # both outside
    before = rng.integers(0, 256, rq.kv_cache_shape(pages, h, D, page), dtype=np.uint8)
    want = before.copy()
    codes, scales = ref.tiles(want, page, D)
    for side, x in enumerate((k, v)):
        o = oracle.run_quant_f32(x.float().numpy().reshape(n * h, D), mode="nvfp4", scale_in=float(gs[side]))
        q, s = o["q"].reshape(n, h, D // 2), o["scales"].reshape(n, h, D // 16)
        for t in range(n):
            if 0 <= slots[t] < pages * page:
                codes[slots[t] // page, side, :, slots[t] % page] = q[t]
                scales[slots[t] // page, side, :, slots[t] % page] = s[t]
    # keys and values as column ranges of one wider buffer
    wide = torch.randn(n, (3 * h + 1) * D).to(DT[dtype])
    wide[:, h * D: 2 * h * D] = k.flatten(1)
    wide[:, 2 * h * D: 3 * h * D] = v.flatten(1)
    wide = wide.cuda()
    dk = wide[:, h * D: 2 * h * D].unflatten(1, (h, D))
    dv = wide[:, 2 * h * D: 3 * h * D].unflatten(1, (h, D))
    cache, ds = torch.from_numpy(before).cuda(), torch.from_numpy(slots).cuda()
    g = [torch.tensor([x], device="cuda") for x in gs]
    rq.kv_cache_store_nvfp4(dk, dv, ds, *g, cache, page)
    assert np.array_equal(cache.cpu().numpy(), want)

    # load, into a buffer with the same interleaved layout
    out = torch.full_like(wide, 7.0)
    ko = out[:, h * D: 2 * h * D].unflatten(1, (h, D))
    vo = out[:, 2 * h * D: 3 * h * D].unflatten(1, (h, D))
    rq.kv_cache_load_nvfp4(cache, ds, *g, D, page, DT[dtype], k_out=ko, v_out=vo)
    for side, o in enumerate((ko, vo)):
        full = np.zeros((n, h, D))
        for t in range(n):
            if 0 <= slots[t] < pages * page:
                p, i = slots[t] // page, slots[t] % page
                full[t] = ref.values(codes[p, side, :, i], scales[p, side, :, i], 1.0)
        # code * scale is exact; one fp32 division, one rounding to T
        exp = torch.from_numpy(full.astype(np.float32) / gs[side]).to(DT[dtype])
        assert torch.equal(o.cpu(), exp)
    assert (out[:, : h * D] == 7).all() and (out[:, 3 * h * D:] == 7).all()
    k2, v2 = rq.kv_cache_load_nvfp4(cache, ds, *g, D, page, DT[dtype])
    assert torch.equal(k2, ko) and torch.equal(v2, vo)


def test_load_reads_nan_scales_as_448(rmsq_gpu):
    cache = torch.full(rmsq_gpu.kv_cache_shape(1, 1, 64, 16), 0xff, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    k, v = rmsq_gpu.kv_cache_load_nvfp4(cache, torch.arange(16, device="cuda"), one, one, 64, 16)
    assert (k == -6 * 448).all() and (v == -6 * 448).all()


def test_store_saturates_and_keeps_infinities_out_of_the_scales(rmsq_gpu):
    """Infinite elements take the largest code; the scale stays finite."""
    k = torch.randn(4, 1, 64, device="cuda").bfloat16()
    k[1, 0, 3], k[2, 0, 5], k[3, 0, 7] = float("inf"), float("-inf"), 3e38
    cache = torch.zeros(rmsq_gpu.kv_cache_shape(1, 1, 64, 16), dtype=torch.uint8, device="cuda")
    gs = torch.tensor([336.0], device="cuda")
    rmsq_gpu.kv_cache_store_nvfp4(k, k, torch.arange(4, device="cuda"), gs, gs, cache, 16)
    scales = ref.tiles(cache.cpu().numpy(), 16, 64)[1]
    assert (scales <= 0x7e).all() and scales[0, 0, 0, 1, 0] == 0x7e
    k2, _ = rmsq_gpu.kv_cache_load_nvfp4(cache, torch.arange(4, device="cuda"), gs, gs, 64, 16)
    assert torch.isfinite(k2).all() and k2[1, 0, 3] == 8.0 and k2[2, 0, 5] == -8.0


def test_cache_on_a_side_stream_and_in_a_graph(rmsq_gpu):
    rq = rmsq_gpu
    rng = np.random.default_rng(3)
    k, v = _kv(rng, 50, 2, 128, "bf16").cuda(), _kv(rng, 50, 2, 128, "bf16").cuda()
    gs = torch.tensor([27.0], device="cuda")
    slots = torch.randperm(64, device="cuda")[:50]
    a = torch.zeros(rq.kv_cache_shape(4, 2, 128, 16), dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    rq.kv_cache_store_nvfp4(k, v, slots, gs, gs, a, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rq.kv_cache_store_nvfp4(k, v, slots, gs, gs, b, 16)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)
    c = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rq.kv_cache_store_nvfp4(k, v, slots, gs, gs, c, 16)
    k.neg_()
    v.add_(1)
    g.replay()
    rq.kv_cache_store_nvfp4(k, v, slots, gs, gs, a, 16)
    torch.cuda.synchronize()
    assert torch.equal(a, c)


def test_cache_offsets_beyond_32_bits(rmsq_gpu):
    """A cache of over 4 GiB: the last page's tokens land there."""
    rq, page, h, D = rmsq_gpu, 256, 8, 128
    pages = (4 << 30) // (2 * h * page * D * 9 // 16) + 3
    cache = torch.zeros(rq.kv_cache_shape(pages, h, D, page), dtype=torch.uint8, device="cuda")
    k = torch.randn(3, h, D, device="cuda").bfloat16()
    gs = torch.tensor([336.0], device="cuda")
    slots = torch.tensor([pages * page - 1, 0, (pages - 1) * page], device="cuda")
    rq.kv_cache_store_nvfp4(k, -k, slots, gs, gs, cache, page)
    k2, v2 = rq.kv_cache_load_nvfp4(cache, slots, gs, gs, D, page)
    small = torch.zeros(rq.kv_cache_shape(1, h, D, page), dtype=torch.uint8, device="cuda")
    three = torch.arange(3, device="cuda")
    rq.kv_cache_store_nvfp4(k, -k, three, gs, gs, small, page)
    k3, v3 = rq.kv_cache_load_nvfp4(small, three, gs, gs, D, page)
    assert torch.equal(k2, k3) and torch.equal(v2, v3) and torch.equal(v2, -k2) and k2.abs().sum() > 0

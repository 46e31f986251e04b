"""The paged FP8 cache's store and load on the GPU: codes and scales have to
equal the plain reference's, byte for byte."""
import numpy as np
import pytest
import torch

import _serve8_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _kv(rng, n, h, D, dtype, spread=4):
    """Tokens of very different strength, some of them zero."""
    x = rng.normal(0, 1, (n, h, D)) * np.exp2(rng.integers(-spread, spread, (n, h, 1)))
    x[rng.random((n, h)) < 0.05] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


def _requests(rng, pages, page, lens):
    """Slots of consecutive positions of requests (context, new tokens) on pages of their own."""
    ids, at, out = rng.permutation(pages), 0, []
    for ctx, new in lens:
        need = -(-(ctx + new) // page)
        mine = ids[at: at + need]
        at += need
        pos = np.arange(ctx, ctx + new)
        out.append(mine[pos // page] * page + pos % page)
    assert at <= pages
    return np.concatenate(out).astype(np.int64) if out else np.zeros(0, np.int64)


def _cache(rng, pages, h, D, page):
    """A filled cache: codes of every value (no NaN), scales around ordinary ones."""
    codes = rng.integers(0, 256, (pages, 2, h, page, D), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    return codes, rng.integers(112, 125, (pages, 2, h, page // 16), dtype=np.uint8)


def _store(rq, codes, scales, k, v, slots, stream=None, view=torch.uint8):
    d_codes, d_scales = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    rq.kv_cache_store_fp8(k, v, torch.from_numpy(slots).cuda(), d_codes.view(view), d_scales, stream=stream)
    torch.cuda.synchronize()
    return d_codes, d_scales


def _check(rq, codes, scales, k, v, slots, **kw):
    want_c, want_s = codes.copy(), scales.copy()
    ref.store(want_c, want_s, k.double().cpu().numpy(), v.double().cpu().numpy(), slots)
    got_c, got_s = _store(rq, codes, scales, k.cuda(), v.cuda(), slots, **kw)
    assert np.array_equal(got_s.cpu().numpy(), want_s)
    # (a NaN's sign is not specified)
    g = got_c.cpu().numpy()
    assert np.array_equal(np.where((g & 127) == 127, 127, g), np.where((want_c & 127) == 127, 127, want_c))
    return got_c, got_s


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h, D, page", [(1, 64, 16), (2, 64, 64), (3, 128, 16), (8, 128, 32), (1, 256, 256), (2, 256, 16)])
@pytest.mark.parametrize("lens", [
    [(0, 1)], [(5, 1)], [(15, 1)], [(16, 1)],                  # first, middle, last slot of a block
    [(0, 16)], [(3, 13)], [(3, 14)], [(31, 33)],               # whole blocks, over their ends
    [(i % 41, 1) for i in range(50)],                          # a decode step
    [(7, 100), (0, 1), (40, 61), (2, 3)],
], ids=lambda v: f"{len(v)}x{v[0][0]}+{v[0][1]}" if isinstance(v, list) else None)
def test_store(rmsq_gpu, dtype, h, D, page, lens):
    rng = np.random.default_rng(D + h + len(lens))
    pages = sum(-(-(c + n) // page) for c, n in lens) + 2
    slots = _requests(rng, pages, page, lens)
    n = len(slots)
    _check(rmsq_gpu, *_cache(rng, pages, h, D, page), _kv(rng, n, h, D, dtype), _kv(rng, n, h, D, dtype), slots)


@pytest.mark.parametrize("n, h", [(5000, 4), (20000, 4), (9000, 8), (7000, 4), (33000, 4)])
def test_store_of_a_prompt(rmsq_gpu, n, h):
    """Sizes for which a warp looks after 2, 4, 8 and 16 tokens; decodes between them."""
    rng = np.random.default_rng(n)
    lens = [(9, n // 2)] + [(i % 30, 1) for i in range(40)] + [(3, n - n // 2 - 40)]
    pages = sum(-(-(c + m) // 64) for c, m in lens) + 2
    slots = _requests(rng, pages, 64, lens)
    _check(rmsq_gpu, *_cache(rng, pages, h, 64, 64), _kv(rng, n, h, 64, "bf16"), _kv(rng, n, h, 64, "bf16"), slots)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_slots_outside_and_padding(rmsq_gpu, dtype):
    """Skipped tokens at the ends and between blocks, slots beyond the cache."""
    rng = np.random.default_rng(3)
    codes, scales = _cache(rng, 5, 2, 128, 32)
    slots = np.array([-1, 3, 4, 160, 37, 38, -5, 1 << 40, 64, 65, 66, 67, -1, -1], np.int64)
    n = len(slots)
    _check(rmsq_gpu, codes, scales, _kv(rng, n, 2, 128, dtype), _kv(rng, n, 2, 128, dtype), slots)


def test_a_block_of_scattered_slots(rmsq_gpu):
    """Ascending slots of one block need not be neighbours."""
    rng = np.random.default_rng(4)
    codes, scales = _cache(rng, 4, 1, 64, 16)
    slots = np.array([2, 5, 6, 15, 16, 31, 48, 50], np.int64)
    _check(rmsq_gpu, codes, scales, _kv(rng, 8, 1, 64, "bf16"), _kv(rng, 8, 1, 64, "bf16"), slots)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_grow_and_stay(rmsq_gpu, dtype, D):
    """A token after another into one block: louder (older codes are rounded,
    down to subnormals and zero), softer, then a fresh block over an old one."""
    rng = np.random.default_rng(D)
    codes = np.full((2, 2, 1, 16, D), 0xff, np.uint8)       # as an unwritten cache may be
    scales = np.full((2, 2, 1, 1), 255, np.uint8)
    loud = [1.0, 0.25, 3.0, 100.0, 90.0, 1.0, 3000.0, 1e-3, 30000.0, 2.0]
    for turn in range(2):
        for o, g in enumerate(loud):
            k = torch.from_numpy(rng.normal(0, 1, (1, 1, D)) * g).to(DT[dtype])
            v = torch.from_numpy(rng.normal(0, 1, (1, 1, D)) / g).to(DT[dtype])
            got_c, got_s = _check(rmsq_gpu, codes, scales, k, v, np.array([16 + o], np.int64))
            codes, scales = got_c.cpu().numpy(), got_s.cpu().numpy()
    assert (codes[0] == 0xff).all() and (scales[0] == 255).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scale_borders(rmsq_gpu, dtype):
    """Maxima at, just above and just below 448 times a power of two, ties of
    the rounding, the smallest and largest scales, zeros."""
    top = [448.0, 450.0, 446.0, 224.0, 3.5, 3.515625, 0.0, 2.0 ** -14]
    if dtype == "bf16":
        top += [448 * 2.0 ** 60, 2.0 ** 100, 1e-12, 448e-12, 1e-30]
    ties = np.array([(1 + (2 * m + 1) / 16) * 2.0 ** e for e in range(-6, 3) for m in range(7)] + [2.0 ** -10, 3 * 2.0 ** -10])
    for t in top:
        x = np.zeros((2, 1, 64))
        x[0, 0, :63] = np.resize(ties, 63) * (t / 448 if t else 0)
        x[1] = -x[0]
        x[0, 0, 63] = t
        k = torch.from_numpy(x).to(DT[dtype])
        _check(rmsq_gpu, np.zeros((1, 2, 1, 16, 64), np.uint8), np.zeros((1, 2, 1, 1), np.uint8), k, k.flip(0),
               np.array([0, 1], np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_not_finite(rmsq_gpu, dtype, D):
    """Infinities and NaN in keys and in values: NaN where they are, NaN in all
    key codes of that token and head, and no effect on the others' scales."""
    rng = np.random.default_rng(D + 1)
    codes, scales = _cache(rng, 3, 2, D, 16)
    k, v = _kv(rng, 20, 2, D, dtype), _kv(rng, 20, 2, D, dtype)
    k[1, 0, 3], k[4, 1, D - 1], v[6, 0, 0], v[7, 0, 5], v[7, 1, 6] = float("nan"), float("inf"), -float("inf"), float("nan"), float("nan")
    k[17], v[18] = float("inf"), float("nan")
    _check(rmsq_gpu, codes, scales, k, v, np.arange(9, 29, dtype=np.int64))
    codes, scales = _cache(rng, 1, 1, D, 16)
    k, v = _kv(rng, 1, 1, D, dtype), _kv(rng, 1, 1, D, dtype)
    v[:] = float("nan")
    _check(rmsq_gpu, codes, scales, k, v, np.array([0], np.int64))      # nothing finite for the scale


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n, h, D, page", [(1, 1, 64, 16), (3, 2, 64, 32), (37, 4, 128, 16), (65, 8, 128, 64), (19, 3, 256, 128),
                                           (2500, 2, 256, 16)])
def test_load(rmsq_gpu, dtype, n, h, D, page):
    """Every code (NaN too) under scales over their whole range, any slots in any
    order, the same one twice, slots outside; columns of one buffer as outputs."""
    rq = rmsq_gpu
    rng = np.random.default_rng(n + D)
    pages = n // page + 3
    codes = rng.integers(0, 256, (pages, 2, h, page, D), dtype=np.uint8)
    scales = rng.integers(0, 256, (pages, 2, h, page // 16), dtype=np.uint8)
    if dtype == "fp16":
        scales = np.clip(scales, 100, 133)
    slots = rng.integers(0, pages * page, n)
    if n > 5:
        slots[2], slots[3], slots[4] = -1, pages * page, slots[5]
    val = ref.values(codes, scales)
    at = np.clip(slots, 0, pages * page - 1)
    inside = (slots >= 0) & (slots < pages * page)
    want = np.where(inside[:, None, None, None], val[at // page, :, :, at % page], 0.0)
    d = [torch.from_numpy(a).cuda() for a in (codes, scales, slots)]
    got = rq.kv_cache_load_fp8(d[0].view(torch.float8_e4m3fn), d[1], d[2], DT[dtype])
    both = torch.zeros(n, 2 * h * D + 8, dtype=DT[dtype], device="cuda")
    cols = both[:, : h * D].unflatten(1, (h, D)), both[:, h * D: 2 * h * D].unflatten(1, (h, D))
    rq.kv_cache_load_fp8(*d, DT[dtype], k_out=cols[0], v_out=cols[1])
    for side in range(2):
        w = torch.from_numpy(want[:, side]).to(DT[dtype])
        for g in (got[side], cols[side]):
            wrong = (g.cpu() != w) & ~(g.cpu().isnan() & w.isnan())
            assert wrong.sum() == 0
    assert (both[:, 2 * h * D:] == 0).all()


def test_store_from_a_qkv_buffer_and_load_what_it_stored(rmsq_gpu):
    """Keys and values as columns of a wider buffer; through build_slot_map, two
    steps of a request; half a step of E4M3 is 2^-4, and 2^-10 of the scale where
    codes are subnormal."""
    rq = rmsq_gpu
    torch.manual_seed(1)
    nq, h, D, page = 4, 2, 128, 32
    cache, scales = (torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(9, h, D, page))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free, left = torch.arange(9, device="cuda").int(), i32([9])
    ctx, kept = i32([0, 0]), []
    for new in ([35, 20], [1, 1], [1, 30]):
        slots, pos, start, seq, left, status = rq.build_slot_map(ctx, i32(new), table, free, left, page, 70)
        qkv = torch.randn(70, (nq + 2 * h) * D, device="cuda").bfloat16()
        heads = qkv.unflatten(1, (nq + 2 * h, D))
        k, v = heads[:, nq: nq + h], heads[:, nq + h:]
        rq.kv_cache_store_fp8(k, v, slots, cache, scales)
        kept.append((slots[: sum(new)], k[: sum(new)], v[: sum(new)]))
        ctx = seq
        assert status.item() == 0
    for slots, k, v in kept:
        for got, x in zip(rq.kv_cache_load_fp8(cache, scales, slots), (k, v)):
            # rounded at most twice (its scale may have grown since)
            assert ((got.float() - x.float()).abs() <= 2 * (x.float().abs() * 2 ** -4 + 2.0 ** -10 * 2.0 ** -6)).all()


def test_offsets_beyond_32_bits(rmsq_gpu):
    """A cache of more than 4 GB."""
    rq = rmsq_gpu
    h, D, page = 8, 256, 256
    pages = (5 << 30) // (2 * h * page * D)
    cache = torch.empty(rq.kv_cache_shapes_fp8(pages, h, D, page)[0], dtype=torch.uint8, device="cuda")
    scales = torch.full(rq.kv_cache_shapes_fp8(pages, h, D, page)[1], 255, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(8)
    slots = np.concatenate([np.arange(16), np.arange(pages * page - 48, pages * page)]).astype(np.int64)
    k, v = _kv(rng, 64, h, D, "bf16").cuda(), _kv(rng, 64, h, D, "bf16").cuda()
    d_slots = torch.from_numpy(slots).cuda()
    rq.kv_cache_store_fp8(k, v, d_slots, cache, scales)
    small = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(4, h, D, 16)]
    rq.kv_cache_store_fp8(k, v, torch.arange(64, device="cuda"), *small)
    for a, b in zip(rq.kv_cache_load_fp8(cache, scales, d_slots), rq.kv_cache_load_fp8(*small, torch.arange(64, device="cuda"))):
        assert torch.equal(a, b)

"""The FP8 cache's store where the tokens of a block are interrupted by skipped
entries of the slot map, and where a warp looks after several of them: codes and
scales byte for byte the plain reference's."""
import numpy as np
import pytest
import torch

import test_gpu_kv_cache_fp8 as kv

pytestmark = pytest.mark.gpu


def _holes(rng, slots, share):
    """Some entries taken out, as -1 or as slots beyond the cache."""
    out = slots.copy()
    gone = rng.random(len(out)) < share
    out[gone] = rng.choice(np.array([-1, -7, 1 << 40], np.int64), gone.sum())
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h, D, page", [(1, 64, 16), (2, 128, 64), (3, 256, 32)])
@pytest.mark.parametrize("slots", [
    [3, -1, 4],                                                         # a hole in a decode's block
    [0, -1, -1, 3],
    [16] + [-1] * 14 + [31],                                            # the first and the last of 16
    [17, -1, 18, 1 << 40, 20, -5, 21, -1, -1, 31, -1, 32, -1, 33],      # over a block's end
    [-1] * 20 + [5, -1, 6] + [-1] * 40 + [40, -1, 41, -1],              # behind long stretches
    [5, -1, 6, 37, -1, 38, 20, -1, 21, 48, -1, -1, 50],                 # four requests
    [9, -1, 25, -1, 41, -1, 57],                                        # another block behind each hole
    list(range(64)),
], ids=str)
def test_runs_with_holes(rmsq_gpu, slots, h, D, page, dtype):
    rng = np.random.default_rng(len(slots) + D)
    slots = np.array(slots, np.int64)
    n = len(slots)
    kv._check(rmsq_gpu, *kv._cache(rng, 64 // page + 1, h, D, page), kv._kv(rng, n, h, D, dtype), kv._kv(rng, n, h, D, dtype), slots)


@pytest.mark.parametrize("share", [0.05, 0.5])
@pytest.mark.parametrize("n, h, D", [(700, 2, 128), (3000, 4, 64), (2200, 8, 128), (7000, 4, 128), (5000, 8, 256), (16500, 8, 64)])
def test_prompts_and_decodes_with_holes(rmsq_gpu, n, h, D, share):
    """Sizes for which a warp looks after 1, 2, 4, 8 and 16 tokens."""
    rng = np.random.default_rng(n + int(10 * share))
    lens = [(9, n // 2)] + [(i % 30, 1) for i in range(40)] + [(3, n - n // 2 - 40)]
    pages = sum(-(-(c + m) // 64) for c, m in lens) + 2
    slots = _holes(rng, kv._requests(rng, pages, 64, lens), share)
    kv._check(rmsq_gpu, *kv._cache(rng, pages, h, D, 64), kv._kv(rng, n, h, D, "bf16"), kv._kv(rng, n, h, D, "bf16"), slots)


@pytest.mark.parametrize("D, dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16")])
@pytest.mark.parametrize("n, h", [(1100, 1), (2500, 8), (5000, 8), (9000, 8), (4200, 32)])
def test_several_runs_of_a_warp(rmsq_gpu, n, h, D, dtype):
    """The same sizes for every head length: prompts, decodes side by side, and
    tokens that are not finite in runs that share a warp with others."""
    rng = np.random.default_rng(n + D)
    lens = [(9, n // 2)] + [(i % 31, 1 + i % 3) for i in range(60)]
    lens.append((3, n - sum(m for _, m in lens)))
    pages = sum(-(-(c + m) // 32) for c, m in lens) + 2
    slots = kv._requests(rng, pages, 32, lens)
    k, v = kv._kv(rng, n, h, D, dtype), kv._kv(rng, n, h, D, dtype)
    odd = rng.choice(n, 40, replace=False)
    odd[:20] = n // 2 + np.arange(20) * 3                   # among the short requests
    for i, t in enumerate(odd):
        x = (k, v)[i % 2]
        x[t, rng.integers(h), rng.integers(D)] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    k[odd[0]] = float("nan")
    kv._check(rmsq_gpu, *kv._cache(rng, pages, h, D, 32), k, v, slots)


def test_a_store_with_holes_gives_the_same_every_time(rmsq_gpu):
    rng = np.random.default_rng(2)
    slots = _holes(rng, kv._requests(rng, 60, 32, [(5, 700), (0, 1), (17, 300), (4, 1)]), 0.4)
    args = (*kv._cache(rng, 60, 4, 128, 32), kv._kv(rng, len(slots), 4, 128, "bf16").cuda(),
            kv._kv(rng, len(slots), 4, 128, "bf16").cuda(), slots)
    first = kv._store(rmsq_gpu, *args)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, kv._store(rmsq_gpu, *args)))


def test_an_interrupted_step_of_a_request(rmsq_gpu):
    """Through build_slot_map, then every third token taken out: what is stored comes back."""
    rq = rmsq_gpu
    torch.manual_seed(1)
    h, D, page = 2, 128, 32
    cache, scales = (torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(12, h, D, page))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    slots, _, _, _, _, status = rq.build_slot_map(i32([0, 0]), i32([100, 61]), table, torch.arange(12, device="cuda").int(),
                                                  i32([12]), page, 170)
    assert status.item() == 0
    # (the first token of each block stays: it is what begins the block)
    drop = (torch.arange(170, device="cuda") % 3 == 1) & (slots % 16 != 0)
    slots = torch.where(drop, torch.full_like(slots, -1), slots)
    k, v = (torch.randn(170, h, D, device="cuda").bfloat16() for _ in range(2))
    rq.kv_cache_store_fp8(k, v, slots, cache, scales)
    live = slots >= 0
    for got, x in zip(rq.kv_cache_load_fp8(cache, scales, slots), (k, v)):
        # half a step of E4M3, and 2^-10 of the scale (at most 2^-6 for values below 7) where codes are subnormal
        assert ((got.float() - x.float()).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -16)[live].all()
        assert (got[~live] == 0).all()

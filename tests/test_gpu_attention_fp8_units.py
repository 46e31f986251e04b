"""Attention over the paged FP8 cache where blocks' value scales are far apart:
what a row holds its weights relative to is what that row sees, weighed, and
nothing else.  Against float64, with tolerances relative to the row's own
contributions (an output of zeros is outside them)."""
import math

import numpy as np
import pytest
import torch

import _serve8_ref as ref
import test_gpu_attention_fp8 as attn

pytestmark = pytest.mark.gpu
VARIANTS = ("direct", "pipelined")


def exact(c, window, variant="direct"):
    """out and lse in float64, and their tolerances.

    With w the exact weights (sum 1), S_j the value scale of key j's block, A = sum
    w |v| and U = max w_j S_j, all over the keys that the row sees:
      - the output's rounding, half a step, and 2^-25 (bf16: 2^-134) among subnormal numbers;
      - weights rounded to f16: half a step is 2^-11 of each, 2^-11 A;
      - they are held so that the largest w_j S_j is 2^5 at least, 2^-1 in the kernel for
        prompts (blocks up to 2^7 apart share the scale of the largest); below 2^-14 f16
        has steps of 2^-24: off by 2^-25 each, 2^-30 U or 2^-24 U, times a code of at
        most 448;
      - logits: D + 8 full steps of 2^-23 of scale sum |q||k|, 2^-21 for the exponential,
        2^-22 |logit| for subtraction and factor, and 2^-16 for the exponent of a value
        scale (up to 186, 2^-24 of it, times ln 2, twice) added to them: ds, which moves
        the output by 2 ds A at most;
      - sums over n keys in fp32: n 2^-23 A each for numerator and denominator.
    lse: ds, n 2^-23, 2^-20 for the logarithm, its own rounding."""
    eps = torch.finfo(attn.DT[c["dtype"]]).eps
    val, sv = ref.values(c["codes"], c["scales"]), ref.scale_values(c["scales"])
    D, page = c["D"], c["page"]
    T, H = sum(c["q_lens"]), c["q64"].shape[1]
    G = H // c["codes"].shape[2]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -math.inf)
    tol, tol_lse = np.zeros((T, H, D)), np.zeros((T, H))
    t = 0
    for r, (m, n) in enumerate(zip(c["q_lens"], c["seq"])):
        at, off = c["table"][r, np.arange(n) // page], np.arange(n) % page
        for h in range(H):
            k, v, s = val[at, 0, h // G, off], val[at, 1, h // G, off], sv[at, 1, h // G, off // 16]
            q = c["q64"][t: t + m, h]
            pos = np.arange(n - m, n)[:, None]
            see = (np.arange(n) <= pos) & ((np.arange(n) > pos - window) if window else True)
            z = np.where(see, q @ k.T / math.sqrt(D), -math.inf)
            top = z.max(1, keepdims=True)
            e = np.exp(z - top)
            total = e.sum(1, keepdims=True)
            w = e / total
            A, U = w @ np.abs(v), (w * s).max(1, keepdims=True)
            seen = np.where(see, np.abs(q) @ np.abs(k).T / math.sqrt(D), 0.0).max(1, keepdims=True)
            ds = (D + 8) * 2.0 ** -23 * seen + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(see, z, 0.0)).max(1, keepdims=True) + 2.0 ** -16
            cnt = see.sum(1, keepdims=True)
            o = w @ v
            out[t: t + m, h], lse[t: t + m, h] = o, (top + np.log(total))[:, 0]
            tol[t: t + m, h] = eps / 2 * np.abs(o) + A * (2.0 ** -11 + 2 * ds + 2 * cnt * 2.0 ** -23) + \
                cnt * 2.0 ** (-30 if variant == "direct" else -24) * 448 * U + (2.0 ** -25 if eps == 2.0 ** -10 else 2.0 ** -134)
            tol_lse[t: t + m, h] = (ds + cnt * 2.0 ** -23 + 2.0 ** -20)[:, 0] + 2.0 ** -23 * np.abs(lse[t: t + m, h])
        t += m
    return out, lse, tol, tol_lse


def check(rq, c, *, window=0, variant="direct"):
    out, lse = attn.run(rq, c, window=window, variant=variant)
    want, w_lse, tol, tol_lse = exact(c, window, variant)
    assert (np.abs(want) > tol).mean() > 0.9, "the tolerance would let zeros pass"
    off = np.abs(out.double().cpu().numpy() - want) - tol
    assert not (off > 0).any() and not np.isnan(off).any(), \
        f"{(off > 0).sum()} of {off.size} beyond, up to {(np.abs(off + tol) / np.abs(want))[off > 0].max():.2g} of the value"
    off = np.abs(lse.double().cpu().numpy() - w_lse) - tol_lse
    assert not (off > 0).any() and not np.isnan(off).any(), f"lse beyond by {np.nanmax(off)}"
    assert rq.take_fault_flags() == 0


def blocks_of(c, r, first, count=1):
    """(page, block in it) of blocks of 16 keys of a request."""
    per = c["page"] // 16
    return [(c["table"][r, b // per], b % per) for b in range(first, first + count)]


def set_block(c, r, block, *, v_byte=None, logit=None):
    """The value scale of a block of keys; its keys as equal numbers whose logits are
    about `logit` (to E4M3's precision) with queries of ones."""
    page, b = blocks_of(c, r, block)[0]
    if v_byte is not None:
        c["scales"][page, 1, :, b] = v_byte
    if logit is not None:
        x = logit / math.sqrt(c["D"])
        e = 0 if x == 0 else math.floor(math.log2(abs(x)))
        c["scales"][page, 0, :, b] = 127 + e
        c["codes"][page, 0, :, 16 * b: 16 * b + 16] = ref.encode(np.array([x * 2.0 ** -e]))[0]


def near_ones(c, seed=0):
    """Queries of 0.9 to 1.1."""
    q = torch.from_numpy(np.random.default_rng(seed).uniform(0.9, 1.1, c["q64"].shape)).to(attn.DT[c["dtype"]])
    c["q"], c["q64"] = q, q.double().numpy()


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("place", [0, 3, -1])
def test_a_loud_block_of_no_weight(rmsq_gpu, D, place, variant):
    """A block with a value scale of 2^60 and logits of about -100 amid ordinary ones, as
    the first, a middle and the last one of its request: nothing of it is in the outputs."""
    c = attn.make([90, 3, 1], [400, 333, 150], 4, 2, D, 16, "bf16", seed=D)
    near_ones(c)
    for r, n in enumerate(c["seq"]):
        set_block(c, r, place % ((n - 1) // 16 + 1), v_byte=187, logit=-100.0)
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D, heads", [(64, 2), (64, 16), (128, 6), (256, 2)])
@pytest.mark.parametrize("window", [1, 5, 16])
def test_loud_blocks_that_only_neighbours_see(rmsq_gpu, D, heads, window, variant):
    """Every third block of value scale 2^60, queries that see one or two blocks: those
    that do not see a loud one give ordinary numbers, whatever shares their tile."""
    c = attn.make([100, 4], [200, 70], heads, 1, D, 32, "bf16", seed=window)
    for r, n in enumerate(c["seq"]):
        for b in range(1, n // 16, 3):
            set_block(c, r, b, v_byte=187)
    check(rmsq_gpu, c, window=window, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_grow_fast_along_the_keys(rmsq_gpu, D, variant):
    """The value scale of a block 2^14 times the one before it: early queries see only
    the small ones."""
    c = attn.make([115], [115], 2, 1, D, 16, "bf16", seed=6)
    for b in range(8):
        set_block(c, 0, b, v_byte=88 + 14 * b)
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("apart", [16, 18, 20, 35])
def test_small_values_of_large_weight(rmsq_gpu, D, dtype, apart, variant):
    """Blocks whose value scales are 2^apart apart in every tile, the larger ones'
    weights smaller by about as much: both count."""
    c = attn.make([80, 2], [300, 210], 4, 2, D, 16, dtype, seed=apart, k_scale=(117, 118), v_scale=(118, 119))
    near_ones(c, apart)
    for r, n in enumerate(c["seq"]):
        for b in range(0, (n - 1) // 16 + 1, 2):
            set_block(c, r, b, v_byte=118 + apart, logit=-apart * math.log(2))
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("apart", [4, 7, 8, 14])
def test_large_values_of_little_weight(rmsq_gpu, D, apart, variant):
    """Every second block's values 2^apart larger and of weight e^-20; where the others'
    are next to nothing (every second dim) it is these that count."""
    c = attn.make([150, 70], [300, 200], 4, 2, D, 16, "bf16", seed=D, k_scale=(117, 118), v_scale=(110, 111))
    near_ones(c)
    c["codes"][:, 1, :, :, 1::2] = 1
    rng = np.random.default_rng(apart)
    for r, n in enumerate(c["seq"]):
        for b in range(1, (n - 1) // 16 + 1, 2):
            set_block(c, r, b, v_byte=110 + apart, logit=-20.0)
            page, at = blocks_of(c, r, b)[0]
            c["codes"][page, 1, :, 16 * at: 16 * at + 16] = rng.integers(0, 127, (2, 16, D)) | 128 * rng.integers(0, 2, (2, 16, D))
    check(rmsq_gpu, c, window=32, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [20.0, 30.0, 100.0])
@pytest.mark.parametrize("least, most", [(88, 120), (88, 187), (60, 187), (1, 187), (1, 2), (1, 100), (40, 41)])
def test_scale_bytes_of_any_size(rmsq_gpu, D, gap, least, most, variant):
    """The least scale where the weight is, the largest everywhere else: the sum of the
    weights counts the former (bytes below 88 are none the store writes)."""
    c = attn.make([90, 1], [200, 150], 4, 1, D, 16, "bf16", seed=least, k_scale=(117, 118), v_scale=(most, most + 1))
    near_ones(c)
    for r in range(2):
        for b in (0, 1, 5):
            set_block(c, r, b, v_byte=least, logit=gap)
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
def test_far_logits_and_far_scales(rmsq_gpu, variant):
    """Logits beyond 2^10, where the maximum is subtracted first, with value scales that
    rise and fall from block to block."""
    c = attn.make([90, 2], [300, 200], 4, 1, 64, 16, "bf16", seed=4, k_scale=(128, 130), v_scale=(100, 101))
    for r, n in enumerate(c["seq"]):
        for b in range((n - 1) // 16 + 1):
            set_block(c, r, b, v_byte=100 + 29 * (b * 5 % 4))
    check(rmsq_gpu, c, variant=variant)


@pytest.mark.parametrize("D, heads, kv", [(64, 8, 8), (128, 12, 4), (256, 6, 2)])
def test_long_contexts_cut_over_the_card(rmsq_gpu, D, heads, kv):
    """Loud blocks of no weight in some of the parts that the second launch joins."""
    c = attn.make([1, 2, 1], [6000, 3000, 700], heads, kv, D, 64, "bf16", seed=D, k_scale=(117, 118))
    near_ones(c)
    for r, n in enumerate(c["seq"]):
        for b in range(2, n // 16, 37):
            set_block(c, r, b, v_byte=187, logit=-100.0)
    check(rmsq_gpu, c)


@pytest.mark.parametrize("D, heads, kv", [(64, 8, 8), (128, 12, 4), (256, 6, 2)])
def test_weights_and_values_in_different_parts(rmsq_gpu, D, heads, kv):
    """The weight in the first parts, whose values are next to nothing; the values in the others."""
    c = attn.make([1, 2, 1], [6000, 3000, 700], heads, kv, D, 64, "bf16", seed=D, k_scale=(115, 116), v_scale=(187, 188))
    near_ones(c)
    for r in range(3):
        for b in range(16):
            set_block(c, r, b, v_byte=1, logit=20.0)
    check(rmsq_gpu, c)

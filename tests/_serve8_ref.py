"""Plain 64-bit references of the operators around the paged FP8 cache: the
rotation with three axes, the cache's store, attention over it.  Numpy float64,
from the definitions; nothing of the library."""
from __future__ import annotations

import math

import numpy as np

E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)])
E4M3 = np.concatenate([E4M3, -E4M3])
E4M3[[127, 255]] = np.nan
LEAST, MOST = 88, 187           # scale bytes of the store


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even one, saturating; NaN for NaN."""
    grid = E4M3[:127]
    m = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(grid, m), 1, 126)
    lo = hi - 1
    up, down = grid[hi] - m, m - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(m == 0, 0, code) + 128 * np.signbit(x)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def scale_byte(amax: float) -> int:
    """Byte of the smallest power of two s with amax / s <= 448, within the store's range."""
    m, e = math.frexp(max(amax / 448.0, 1e-12))
    return min((e - 1 if m == 0.5 else e) + 127, MOST)


def store(codes, scales, k, v, slots):
    """The store on uint8 arrays codes [pages, 2, heads, page, D] and scales
    [pages, 2, heads, page / 16], in place; k, v float64 [n, heads, D]."""
    pages, _, heads, page, D = codes.shape
    blocks = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            blocks.setdefault(int(s) // 16, []).append((t, int(s) % 16))
    for b, members in blocks.items():
        pg, at = divmod(b * 16, page)
        fresh = members[0][1] == 0
        taken = [o for _, o in members]
        for h in range(heads):
            toks = [t for t, _ in members]
            bad = ~np.isfinite(k[toks, h]).all(-1) | ~np.isfinite(v[toks, h]).all(-1)
            for side, x in ((0, k), (1, v)):
                x = x[toks, h]
                finite = np.abs(x[np.isfinite(x)])
                e = scale_byte(finite.max() if finite.size else 0.0)
                row = codes[pg, side, h, at: at + 16]
                if not fresh:
                    had = min(max(int(scales[pg, side, h, at // 16]), 1), MOST)
                    if e > had:
                        keep = [o for o in range(16) if o not in taken]
                        row[keep] = encode(E4M3[row[keep]] * 2.0 ** (had - e))
                    e = max(e, had)
                y = np.where(np.isfinite(x), x, np.nan)
                if side == 0:
                    y = np.where(bad[:, None], np.nan, y)
                row[taken] = encode(y * 2.0 ** (127 - e))
                scales[pg, side, h, at // 16] = e


def scale_values(scales: np.ndarray) -> np.ndarray:
    return np.exp2(np.clip(scales.astype(np.float64), 1, MOST) - 127)


def values(codes, scales):
    """Elements [pages, 2, heads, page, D] of a cache."""
    return E4M3[codes] * np.repeat(scale_values(scales), 16, -1)[..., None]


def axes(half, sections, interleaved):
    t, h, w = sections
    i = np.arange(half)
    if interleaved:
        return np.where((i % 3 == 1) & (i < 3 * h), 1, np.where((i % 3 == 2) & (i < 3 * w), 2, 0))
    return np.where(i < t, 0, np.where(i < t + h, 1, 2))


def rotate(x, pos, table, q_w, k_w, eps, nq, sections, interleaved, neox):
    """x float64 [n, heads, D] (q heads first): result, and the bound of the
    fp32 steps' error.  A sum of D squares by a tree adds log2(D) + 1 roundings,
    then the mean, eps, square root, reciprocal, two products: at most 16 half
    steps of 2^-24 in all on a normed element; two products, a sum: 3 more, each
    relative to the pair's magnitude |a| + |b| (cos and sin are at most 1)."""
    n, heads, D = x.shape
    half = D // 2
    if q_w is not None:
        w = np.concatenate([np.broadcast_to(q_w, (nq, D)), np.broadcast_to(k_w, (heads - nq, D))])
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    ax = axes(half, sections, interleaved)
    live = ((pos >= 0) & (pos < len(table))).all(0)
    row = np.where(live, pos, 0)[ax].T                      # [n, half]
    c, s = table[row, np.arange(half)][:, None], table[row, half + np.arange(half)][:, None]
    a, b = (x[..., :half], x[..., half:]) if neox else (x[..., 0::2], x[..., 1::2])
    y, mag = np.empty_like(x), np.empty_like(x)
    for dst, val in ((y, (a * c - b * s, b * c + a * s)), (mag, (np.abs(a) + np.abs(b),) * 2)):
        if neox:
            dst[..., :half], dst[..., half:] = val
        else:
            dst[..., 0::2], dst[..., 1::2] = val
    return y, mag * 20 * 2.0 ** -24, live


def attention(q, codes, scales, table, q_lens, seq_lens, softmax_scale, window, eps):
    """out, lse in float64 and their tolerances.

    Per output element, with p the exact weights (sum 1) and A = sum p |v|:
      - the output's rounding, half a step: eps / 2 |out|, and among fp16's
        subnormal numbers (below 2^-14, steps of 2^-24) 2^-25;
      - weights rounded to f16: 2^-11 A; they are held relative to the largest
        value scale S of the request's head, the largest of them as 2^5 at least,
        and where that product is below 2^-19 of it it is subnormal in f16, off by
        2^-25 (half a step), so 2^-30 of it, times a code of at most 448:
        n 2^-30 448 S;
      - logits: a dot product of D exact products summed in fp32, counted with
        a full step (2^-23) per addition because the matrix unit may truncate:
        ds = (D + 8) 2^-23 scale sum|q||k|, 2^-21 for the exponential and
        2^-22 |logit| for the rounding of subtraction and factor (the scales of
        the keys are powers of two, exact); a relative change ds of every weight
        moves the output by at most 2 ds A;
      - fp32 sums over n keys: n 2^-23 A each for numerator and denominator.
    lse: ds, the fp32 sum of the weights n 2^-23 and 2^-20 for the logarithm,
    plus its own rounding."""
    T, H, D = q.shape
    pages, _, kv, page, _ = codes.shape
    val = values(codes, scales) if pages else np.zeros((1, 2, kv, page, D))
    sv = scale_values(scales) if pages else np.ones((1, 2, kv, page // 16))
    out, lse = np.zeros((T, H, D)), np.full((T, H), -math.inf)
    tol, tol_lse = np.zeros((T, H, D)), np.zeros((T, H))
    t = 0
    G = H // kv
    for r, (m, n) in enumerate(zip(q_lens, seq_lens)):
        idx = np.array([int(table[r][j // page]) for j in range(n)], np.int64)
        ok = (idx >= 0) & (idx < pages)
        at, off = np.where(ok, idx, 0), np.arange(n) % page
        for i in range(m):
            p = n - m + i
            see = ok & (np.arange(n) <= p)
            if window:
                see &= np.arange(n) > p - window
            if see.any():
                a, o = at[see], off[see]
                for h in range(H):
                    kk, vv = val[a, 0, h // G, o], val[a, 1, h // G, o]
                    vv = np.where(np.isnan(vv), 448.0 * sv[a, 1, h // G, o // 16][:, None], vv)
                    s = kk @ q[t, h] * softmax_scale
                    mx = s.max()
                    e = np.exp(s - mx)
                    w = e / e.sum()
                    out[t, h] = w @ vv
                    lse[t, h] = mx + math.log(e.sum()) if not np.isnan(mx) else np.nan
                    A = w @ np.abs(vv)
                    ds = ((D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[t, h])) * softmax_scale).max() + \
                        2.0 ** -21 + 2.0 ** -22 * np.abs(s).max()
                    cnt = len(s)
                    big = sv[at[ok], 1, h // G, off[ok] // 16].max()
                    tol[t, h] = eps / 2 * np.abs(out[t, h]) + A * (2.0 ** -11 + 2 * ds + 2 * cnt * 2.0 ** -23) + \
                        cnt * 2.0 ** -30 * 448 * big + (2.0 ** -25 if eps == 2.0 ** -10 else 0.0)
                    tol_lse[t, h] = ds + cnt * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -23 * abs(lse[t, h])
            t += 1
    return out, lse, tol, tol_lse

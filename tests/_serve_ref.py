"""Plain 64-bit references of the serving operators: slot maps, the paged
NVFP4 cache format, attention over it.  Python integers and numpy / torch
float64, from the definitions; nothing of the library."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3_table() -> np.ndarray:
    """Value of each scale byte; the NaN codes read as 448."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = 448.0 if (c & 127) == 127 else -v if c & 128 else v
    return out


E4M3 = e4m3_table()


def slot_map(ctx, qlen, table, free, num_free, page, max_tokens):
    """The definition, request by request.  Returns (slots, positions, start,
    seq, num_free_out, status, table)."""
    R, width = table.shape
    table = table.copy()
    status = 0
    if any(c < 0 or q < 0 for c, q in zip(ctx, qlen)) or not 0 <= num_free <= len(free):
        status |= 8
    ok = [(c, q) for c, q in zip(ctx, qlen) if c >= 0 and q >= 0]
    need = [-(-(c + q) // page) - -(-c // page) for c, q in ok]
    if 0 <= num_free <= len(free) and sum(need) > num_free:
        status |= 1
    if any(-(-(c + q) // page) > width for c, q in ok):
        status |= 2
    if sum(q for _, q in ok) > max_tokens:
        status |= 4
    slots, pos = [-1] * max_tokens, [-1] * max_tokens
    if status:
        return slots, pos, [0] * (R + 1), list(ctx), num_free, status, table
    start, left, t = [0], num_free, 0
    for r in range(R):
        for k in range(-(-ctx[r] // page), -(-(ctx[r] + qlen[r]) // page)):
            left -= 1
            table[r, k] = free[left]
        for i in range(qlen[r]):
            p = ctx[r] + i
            pg = int(table[r, p // page])
            pos[t], slots[t] = p, -1 if pg < 0 else pg * page + p % page
            t += 1
        start.append(t)
    return slots, pos, start, [c + q for c, q in zip(ctx, qlen)], left, 0, table


def tiles(cache: np.ndarray, page: int, D: int):
    """Codes [pages, 2, heads, page, D/2] and scale bytes [.., page, D/16] of a cache."""
    n = page * D // 2
    return (cache[..., :n].reshape(*cache.shape[:3], page, D // 2),
            cache[..., n:].reshape(*cache.shape[:3], page, D // 16))


def values(codes: np.ndarray, scales: np.ndarray, gs: float) -> np.ndarray:
    q = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    return q * np.repeat(E4M3[scales], 16, -1) / gs


def request_kv(cache, table_row, seq, page, D, k_gs, v_gs):
    """K, V [heads, seq, D] of a request in float64 and which keys lie on a page of the cache."""
    codes, scales = tiles(cache, page, D)
    idx = [int(table_row[j // page]) for j in range(seq)]
    ok = np.array([0 <= p < cache.shape[0] for p in idx], bool)
    at = np.array([p if g else 0 for p, g in zip(idx, ok)], int)
    off = np.arange(seq) % page
    if cache.shape[0] == 0 or seq == 0:
        return np.zeros((cache.shape[2], seq, D)), np.zeros((cache.shape[2], seq, D)), ok
    k = values(codes[at, 0, :, off], scales[at, 0, :, off], k_gs).transpose(1, 0, 2)
    v = values(codes[at, 1, :, off], scales[at, 1, :, off], v_gs).transpose(1, 0, 2)
    return k, v, ok


def attention(q, cache, table, q_lens, seq_lens, k_gs, v_gs, page, scale, window, eps):
    """out, lse in float64 and their tolerances.

    Per output element, with p the exact weights (sum 1) and A = sum p |v|:
      - the output's rounding, half a step: eps/2 |out|;
      - weights rounded to f16: 2^-11 A; those below 2^-23 of the largest are
        subnormal there, off by 2^-34 of it each: n 2^-34 max|v|;
      - logits: a dot product of D exact products summed in fp32, counted with
        a full step (2^-23) per addition because the matrix unit may truncate:
        ds = (D + 8) 2^-23 scale sum|q||k|, and 2^-21 for the exponential and
        the subtraction's rounding 2^-23 |logit|; a relative change ds of every
        weight moves the output by at most 2 ds A;
      - fp32 sums over n keys: n 2^-23 A each for numerator and denominator.
    lse: ds, the fp32 sum of the weights n 2^-23 and 2^-20 for the logarithm,
    plus its own rounding."""
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -math.inf)
    tol, tol_lse = np.zeros((T, H, D)), np.zeros((T, H))
    t = 0
    for r, (m, n) in enumerate(zip(q_lens, seq_lens)):
        k, v, ok = request_kv(cache, table[r], n, page, D, k_gs, v_gs)
        G = H // k.shape[0]
        for i in range(m):
            p = n - m + i
            see = ok & (np.arange(n) <= p)
            if window:
                see &= np.arange(n) > p - window
            if see.any():
                for h in range(H):
                    kk, vv = k[h // G][see], v[h // G][see]
                    s = kk @ q[t, h] * scale
                    mx = s.max()
                    e = np.exp(s - mx)
                    w = e / e.sum()
                    out[t, h] = w @ vv
                    lse[t, h] = mx + math.log(e.sum())
                    A = w @ np.abs(vv)
                    ds = ((D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[t, h])) * scale).max() + \
                        2.0 ** -21 + 2.0 ** -23 * np.abs(s).max()
                    cnt = len(s)
                    tol[t, h] = eps / 2 * np.abs(out[t, h]) + A * (2.0 ** -11 + 2 * ds + 2 * cnt * 2.0 ** -23) + \
                        cnt * 2.0 ** -34 * np.abs(vv).max()
                    tol_lse[t, h] = ds + cnt * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -23 * abs(lse[t, h])
            t += 1
    return out, lse, tol, tol_lse


def random_cache(rng, pages, heads, page, D, gs_amax=6.0):
    """A cache of codes and scales drawn over their whole range (scale bytes
    0x00 .. 0x7e, centred on ordinary ones), uint8."""
    cache = rng.integers(0, 256, (pages, 2, heads, page * D * 9 // 16), dtype=np.uint8)
    n = page * D // 2
    sc = np.clip(rng.normal(0x50, 12, cache[..., n:].shape), 0, 0x7e).astype(np.uint8)
    cache[..., n:] = sc
    return cache


def act(x: np.ndarray, dtype: torch.dtype):
    """x rounded to dtype: (CPU tensor, its float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    return t, t.double().numpy()

"""64-bit restatement of the 4-bit cache, its attention, the accumulated
weights and the eviction (numpy, loops over heads), and the tolerances of the
GPU tests, derived from the roundings that the kernels make."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def nearest_index(x, grid):
    """Index of the grid point nearest to each x >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def stored(x):
    """The values the cache holds for rows x [..., d] (float64; NaN for a
    block with an infinity or a NaN)."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    amax = np.abs(blocks).max(-1, keepdims=True)
    fine = np.isfinite(amax)
    s = E4M3[nearest_index(np.where(fine, amax, 0.0) / 6, E4M3)]
    y = np.where((s > 0) & fine, np.abs(np.where(fine, blocks, 0.0)) / np.where(s > 0, s, 1.0), 0.0)
    out = np.sign(np.where(fine, blocks, 1.0)) * LEVELS[nearest_index(y, LEVELS)] * s
    return np.where(fine, out, np.nan).reshape(x.shape)


def unpack(codes, scales):
    """Values (float64) of packed rows."""
    codes = codes.astype(np.int64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.concatenate([LEVELS, -LEVELS])[c]
    b = scales.astype(np.int64) & 0x7F
    s = np.concatenate([E4M3, [np.nan]])[b]
    return v * np.repeat(s, 16, -1)


def attend(q, k, v, lengths, scale, causal):
    """q [B, H, Nq, d], k, v [B, Hkv, C, d], float64.  Returns O, lse, the
    weights added per slot [B, Hkv, C], and for the tolerances sum p |v| and
    the largest scale * sum |q| |k| of each row."""
    B, H, Nq, d = q.shape
    Hkv, C = k.shape[1:3]
    o, av = np.zeros_like(q), np.zeros_like(q)
    lse, big = np.full((B, H, Nq), -np.inf), np.zeros((B, H, Nq))
    w = np.zeros((B, Hkv, C))
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            for i in range(Nq):
                n = lengths[b] - (Nq - 1 - i if causal else 0)
                if n <= 0:
                    continue
                s = (k[b, g, :n] @ q[b, h, i]) * scale
                big[b, h, i] = np.max(np.abs(k[b, g, :n]) @ np.abs(q[b, h, i])) * abs(scale)
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, i] = m + np.log(p.sum())
                p /= p.sum()
                o[b, h, i] = p @ v[b, g, :n]
                av[b, h, i] = p @ np.abs(v[b, g, :n])
                w[b, g, :n] += p
    return o, lse, w, av, big


def score_error(big, d):
    """Bound of a score's error in fp32: d products added in any order, the
    factor, the subtraction and the reference, each within 2^-24 relatively
    of sums no larger than `big`."""
    return (d + 16) * 2.0 ** -24 * big


def tol_out(o, av, big, n, vmax, d, dtype):
    """O: the output's own rounding (half a step), the weights' rounding to
    fp16 (2^-11 of each, in numerator and denominator), the scores' error as a
    relative one of each weight (both again), fp16's underflow (2^-25 of a
    weight scaled to at least 2^7, per key), and 2^-20 for sums and
    exponentials."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    rel = 2 * 2.0 ** -11 + 2 * score_error(big, d)[..., None] + 2.0 ** -20
    return half * np.abs(o) + (1 + half) * (rel * (av + np.abs(o)) + n * 2.0 ** -32 * vmax) + 2.0 ** -24


def tol_lse(lse, big, d):
    """lse: the scores' error, the exponentials' and sums' (2^-20), its own rounding."""
    return score_error(big, d) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def tol_weight(w, big, lse, d, w_in=0.0):
    """A weight is exp(score - lse): both errors are relative to it."""
    rel = 2 * score_error(big.max(), d) + 2.0 ** -19 + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0)).max()
    return w * rel + 2.0 ** -23 * (np.abs(w_in) + w) + 1e-30


def select(weight, pos, n, seen, keep, sinks, recent):
    """src of one head (fa_kv4_evict): list of length min(n, keep)."""
    new = min(n, keep)

    def order(j):
        if (sinks > 0 or recent > 0) and (pos[j] < sinks or pos[j] >= seen - recent):
            return (0, j)  # any two of these: the lower slot first
        w = weight[j]
        return (1, -np.inf if np.isnan(w) else -w, not np.isnan(w), j)

    kept = set(sorted(range(n), key=order)[:new])
    late = iter(sorted(j for j in kept if j >= new))
    return [j if j in kept else next(late) for j in range(new)]

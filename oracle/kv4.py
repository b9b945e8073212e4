"""Float64 oracle of the KV cache held in 4 bits: the format, and what each call makes of it.

A row is 128 values 2^exp * s * c with c an e2m1 and s an e4m3 number (one for 16 values); rounding is
to nearest, to the even code at a tie.  The pages have no counterpart of this cache.
"""
from __future__ import annotations

import numpy as np

from .verify import ancestors

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite e4m3 numbers without sign, by their byte
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def nearest(x, grid):
    """Index of the grid number nearest to each |x| (saturated); ties to the even index."""
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.searchsorted(grid, a).clip(1, len(grid) - 1)
    lo = hi - 1
    d_lo, d_hi = a - grid[lo], grid[hi] - a
    return np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)


def round_rows(x, exp):
    """x [..., 128] -> codes [..., 64], scales [..., 8] (bytes).  A NaN counts as 0."""
    x = np.where(np.isnan(x), 0.0, np.asarray(x, np.float64)) * 2.0 ** -exp
    blocks = x.reshape(*x.shape[:-1], 8, 16)
    scale = nearest(np.abs(blocks).max(-1) / 6, E4M3).astype(np.uint8)
    s = E4M3[scale][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(s > 0, np.minimum(np.abs(blocks) / np.where(s > 0, s, 1), 8.0), 0.0)
    # |x| = s * border exactly where the quotient is a tie: neither operand has more than 8 bits
    code = np.where(s > 0, nearest(ratio, E2M1) + 8 * np.signbit(blocks), 0).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def values(codes, scales, exp):
    """Cache rows -> float64 [..., 128].  Every byte stands for a finite value: the sign of a scale byte
    does not count, and 0x7F stands for 480."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 8, 16)
    s = np.append(E4M3, 480.0)[scales & 127]
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7] * s[..., None] * 2.0 ** exp
    return v.reshape(*codes.shape[:-1], 128)


def visible(parent, T, i):
    """Tree slots that node i sees: its ancestors and itself (parent None: a chain)."""
    return list(range(i + 1)) if parent is None else ancestors(parent, i)


def attend(q, k, v, scale, sets):
    """q [T][Hq][128], k, v [keys][Hkv][128], sets[i] the keys that row i sees -> out, lse, and the mean
    magnitude of the values under the same weights (what a relative error of a weight moves out by)."""
    T, Hq, hd = q.shape
    G = Hq // k.shape[1]
    out, size, lse = np.zeros((T, Hq, hd)), np.zeros((T, Hq, hd)), np.full((T, Hq), -np.inf)
    for i in range(T):
        idx = np.asarray(sets[i], int)
        if not len(idx):
            continue
        for h in range(Hq):
            x = k[idx, h // G] @ q[i, h] * scale
            m = x.max()
            p = np.exp(x - m)
            lse[i, h] = m + np.log(p.sum())
            out[i, h] = p @ v[idx, h // G] / p.sum()
            size[i, h] = p @ np.abs(v[idx, h // G]) / p.sum()
    return out, lse, size


def weights(q, lse, k, scale, score, length, rows, decay=1.0):
    """score [Hkv][cap] -> the score after rows (nodes of q, in order) voted; they own the last slots."""
    n = len(rows)
    base = length - n
    G = q.shape[1] // k.shape[1]
    out = score.astype(np.float64).copy()
    out[:, :base] *= decay
    out[:, base:length] = 0
    for j, node in enumerate(rows):
        for h in range(q.shape[1]):
            if lse[node, h] == -np.inf:
                continue
            out[h // G, :base + j + 1] += np.exp(k[:base + j + 1, h // G] @ q[node, h] * scale - lse[node, h])
    return out


def evict(score, length, budget, n_sink, n_recent):
    """Slots of one (layer, sequence, kv head) that stay, ascending."""
    if length <= budget:
        return list(range(length))
    def rank(i):
        s = float(score[i])
        if i < n_sink or i >= length - n_recent:
            return (0, 0.0, i)
        return (2, 0.0, i) if np.isnan(s) else (1, -s, i)
    return sorted(sorted(range(length), key=rank)[:budget])

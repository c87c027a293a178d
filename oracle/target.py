"""The target's verification pass: a paged K/V cache, the attention of a ragged
batch's rows over it, and the rules on the target's scores.

Float64 NumPy from the definitions, a loop for every row, with rounding to bf16
(and to the 4-bit cache's values) exactly where the cache and the outputs are
stored.
"""
from __future__ import annotations

import numpy as np

from .dflash import round_bf16

__all__ = [
    "E2M1",
    "e4m3_values",
    "fp4_values",
    "quantise_fp4",
    "rotate",
    "sees",
    "paged_attention",
    "count_tokens",
    "logit_rules",
]

#: magnitudes of the eight e2m1 codes
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The 256 e4m3 values by byte: sign, four exponent bits (bias 7), three of
    mantissa; 0x7f and 0xff are NaN, there is no infinity."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0**-6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


def _nearest(x, grid):
    """Index of the grid value nearest to each x >= 0 (ties to the even index)."""
    x = np.minimum(x, grid[-1])
    j = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = grid[j - 1], grid[j]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (j % 2 == 0))
    return np.where(up, j, j - 1)


def quantise_fp4(y):
    """Rows of bf16 values [..., d] to (codes uint8 [..., d] of 0..15, scale bytes
    [..., d / 16]): scale = e4m3(max / 6) at most 448, code = e2m1(y / scale)."""
    g = np.asarray(y, dtype=np.float64).reshape(*y.shape[:-1], -1, 16)
    grid = e4m3_values()[:127]
    byte = _nearest(np.abs(g).max(-1) / 6.0, grid)
    s = grid[byte][..., None]
    code = np.where(s > 0, _nearest(np.abs(g) / np.where(s > 0, s, 1.0), E2M1), 0)
    code = code + 8 * np.signbit(g)
    return code.reshape(y.shape).astype(np.uint8), byte.astype(np.uint8)


def fp4_values(codes, scales):
    """The values of codes [..., d] under scale bytes [..., d / 16]."""
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return mag * np.repeat(e4m3_values()[scales], 16, axis=-1)


def rotate(x, cos, sin):
    """Rotate-half of rows x [..., d] by angles of cos, sin [..., d / 2], to bf16."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return round_bf16(np.concatenate([a * cos - b * sin, b * cos + a * sin], -1))


def sees(C, n, j, slot, mode, window, sinks, pos, tree=None):
    """Whether row j of a stream (C committed slots, n rows, positions pos[0..n-1])
    sees `slot`. mode "causal", "block" or "tree" (tree: bool [n][n])."""
    if slot < 0 or slot >= C + n:
        return False
    m = slot - C
    if m >= 0:
        if mode == "causal" and m > j:
            return False
        if mode == "tree" and not tree[j][m]:
            return False
    at = slot if m < 0 else pos[m]
    return window == 0 or pos[j] - at < window or slot < sinks


def paged_attention(q, k, v, C, mode, window, sinks, pos, tree=None, scale=None):
    """Attention of one stream: q [n, nq, d], k, v [C + n, nkv, d] -> (out [n, nq, d]
    unrounded, mass [n, nq, d] = sum of weight * |v|, spread [n, nq] = scale *
    max_c sum_d |q||k_c|): the last two size the rounding errors."""
    n, nq, d = q.shape
    nkv = k.shape[1]
    G = nq // nkv
    scale = d**-0.5 if scale is None else scale
    out, mass, spread = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, nq))
    for j in range(n):
        s = [c for c in range(C + n) if sees(C, n, j, c, mode, window, sinks, pos, tree)]
        if not s:
            continue
        for h in range(nkv):
            kk, vv = k[s, h], v[s, h]
            for g in range(h * G, h * G + G):
                x = kk @ q[j, g] * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[j, g] = w @ vv
                mass[j, g] = w @ np.abs(vv)
                spread[j, g] = scale * (np.abs(kk) @ np.abs(q[j, g])).max()
    return out, mass, spread


def count_tokens(counts, tokens, prompt):
    """Add tokens of one stream to counts (uint16 [V]): bit 15 for a prompt's, else
    one to the count, at most 32767. Ids outside [0, V) are skipped."""
    for t in tokens:
        if not 0 <= t < len(counts):
            continue
        if prompt:
            counts[t] |= 0x8000
        elif counts[t] & 0x7FFF < 0x7FFF:
            counts[t] += 1
    return counts


def logit_rules(x, counts, path_tokens, repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row's scores x [V] (float64 of bf16) under the rules. counts: uint16 [V]
    or None; path_tokens: the drafted tokens on the row's path without the root;
    bias: (id, value) pairs; allowed: bool [V]. Unrounded."""
    x = np.array(x, dtype=np.float64)
    V = len(x)
    count, prompt = np.zeros(V), np.zeros(V, dtype=bool)
    if counts is not None:
        count = (counts & 0x7FFF).astype(np.float64)
        prompt = (counts & 0x8000) != 0
        for t in path_tokens:
            if 0 <= t < V:
                count[t] += 1
    for v in np.nonzero(prompt | (count > 0))[0]:
        x[v] = x[v] / repetition if x[v] > 0 else x[v] * repetition
        if count[v] > 0:
            x[v] -= frequency * count[v] + presence
    for i, b in bias:
        if 0 <= i < V:
            x[i] += b
    if allowed is not None:
        x[~allowed] = -np.inf
    return x

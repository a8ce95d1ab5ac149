"""Plain 64-bit forms of the dense grouped-head operators, and the error that
their kernels' roundings may cause.

Attention of one query row, keys j <= pos: s_j = scale q.k_j, p = softmax(s),
out = sum p_j v_j.  Roundings of the kernels, each at most half a step
(bf16: 2^-8 of the value; fp32: 2^-24):
  - every weight p_j to bf16 (or f16, finer): sum_j 2^-8 p_j |v_j|;
  - the result to bf16: 2^-8 |out|;
  - a score's fp32 sum of D exact products: D 2^-24 scale sum_d |q_d k_d|, and
    a few roundings of it (the scale's, the subtraction of the reference m):
    8 * 2^-24 (|s| + |m|), log2 units; it changes p_j by that much, relatively;
  - fp32 sums of n weights and of n products: n 2^-24 of the sum, counted as
    n / 16 + 64 additions in a row (a lane adds every 16th key or fewer).
"""

from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def rows_of(table, page, base, b, n):
    """Physical rows of the first n tokens of sequence b (CPU int64)."""
    j = torch.arange(n)
    if table is None:
        return int(base[b]) + j
    return table[b, j // page].long() * page + j % page


def values(cache, scale):
    """fp64 values of a cache [rows, heads, d]: bf16, or e4m3 codes with scales [rows, heads]."""
    if scale is None:
        return cache.double()
    return cache.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def attend(q, k, v, pos, sm_scale):
    """q [t, hq, d], k and v [n, hkv, d] in fp64, pos [t] (-1: no key).  Returns out, lse and the
    allowed errors of both."""
    t, hq, d = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    out = torch.zeros(t, hq, d, dtype=torch.float64)
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    eps = 2.0 ** -24
    for i in range(t):
        m = int(pos[i]) + 1
        if m <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h // g], v[:m, h // g]
            s = sm_scale * (kk @ q[i, h])
            top = torch.logsumexp(s, 0)
            p = torch.exp(s - top)
            mag = abs(sm_scale) * (kk.abs() @ q[i, h].abs())
            score = float(eps * (d * mag + 8 * 1.4427 * (s.abs() + s.abs().max())).max())
            adds = eps * (m / 16 + 64)
            av = p @ vv.abs()
            out[i, h] = p @ vv
            lse[i, h] = top
            tol[i, h] = 2.0 ** -8 * out[i, h].abs() + (2.0 ** -8 + 2 * score + 2 * adds) * av
            ltol[i, h] = 2 * score + adds + 8 * eps * (1 + abs(float(top)))
    return out, lse, tol, ltol


def rotate(x, pos, inv_freq, rot, halves):
    """x [n, heads, d] in fp64 with its first rot dims rotated."""
    if inv_freq is None:
        return x.clone()
    y = x.clone()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if halves else (2 * i, 2 * i + 1)
        ang = pos.double() * float(inv_freq[i])
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def quantise(x):
    """(value / scale in fp64, scale) per row of the last axis: scale = amax / 448, 1 for a zero row."""
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return x / scale[..., None], scale

"""Plain forms of the 8-bit cache with a scale per block of tokens and head,
and of the step's plan: request by request, block by block, on the CPU.

An e4m3 code of a value x under a scale s is x / s rounded to nearest even,
saturating at 448; s is a power of two, so x / s is exact in fp64 and its code
is the code of the exact quotient."""

from __future__ import annotations

import math

import torch

import gqa_reference as R

LEAST = 2.0 ** -60


def code_of(x):
    """e4m3 codes (uint8) of fp64 values that are exact in fp32 or were rounded to it."""
    y = x.float().clamp(-448.0, 448.0)  # NaN stays NaN
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def value_of(code):
    return code.view(torch.float8_e4m3fn).double()


def need_of(amax: float) -> float:
    """2^ceil(log2(amax / 448)), at least 2^-60, without a logarithm."""
    if not amax > 448.0 * LEAST:
        return LEAST
    m, e = math.frexp(amax / 448.0)  # in fp64: exact enough, 448 2^k / 448 is exact
    return math.ldexp(1.0, e - 1 if m == 0.5 else e)


def insert(y, code, scale, rows, p0, sb):
    """y [n, heads, d] (fp64) at positions p0 .. of a sequence whose token j is physical row rows[j]:
    codes [rows, heads, d] and scales [rows / sb, heads] changed in place."""
    n = y.shape[0]
    for lo in range(p0 // sb * sb, p0 + n, sb):
        first, last = max(lo, p0), min(lo + sb, p0 + n)
        home = int(rows[lo]) // sb
        for h in range(y.shape[1]):
            part = y[first - p0:last - p0, h]
            finite = part[torch.isfinite(part)]
            s = need_of(float(finite.abs().max()) if finite.numel() else 0.0)
            if first > lo:
                held = float(scale[home, h])
                if held >= s:
                    s = held
                else:
                    old = rows[lo:first]
                    code[old, h] = code_of(value_of(code[old, h]) * (held / s))
            scale[home, h] = s
            code[rows[first:last], h] = code_of(part / s)


def plan(cached, new, page, free, free_range, num_pages, table, num_q):
    """dsa_step_plan on Python lists; table: list of lists, changed in place.  Returns a dict, and
    whether something was refused."""
    width = len(table[0]) if table else 0
    lo, hi = free_range
    bad = not 0 <= lo <= hi <= len(free)
    if bad:
        lo = hi = 0
    at, row, want = lo, 0, 0
    ctx, start, pos, slot = [], [], [-1] * num_q, [-1] * num_q
    for b, (p, n) in enumerate(zip(cached, new)):
        start.append(min(row, num_q))
        rows = max(n, 0)
        ok = p >= 0 and n >= 0 and p + n <= width * page and row + rows <= num_q
        need = -(-(p + n) // page) - -(-p // page) if ok else 0
        if ok and need and want + need > hi - lo:
            ok = False
        if ok:
            for c in range(need):
                table[b][-(-p // page) + c] = free[lo + want + c]
            if need:
                at = lo + want + need
            for i in range(n):
                j = p + i
                pg = table[b][j // page]
                if 0 <= pg < num_pages:
                    pos[row + i], slot[row + i] = j, pg * page + j % page
                else:
                    bad = True
        bad = bad or not ok
        ctx.append(max(0, p + n if ok else p))
        want += need
        row += rows
    start.append(min(row, num_q))
    nxt = [at if 0 <= free_range[0] <= free_range[1] <= len(free) else free_range[0], free_range[1]]
    return dict(ctx=ctx, q_start=start, q_pos=pos, slot=slot, next=nxt, table=table), bad


rotate = R.rotate

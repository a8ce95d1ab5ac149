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
        ok = p >= 0 and n >= 0 and p + n <= min(width * page, 1 << 30) and row + rows <= num_q
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


# ---- blocks chosen by a bound of their scores
def step_of(amax: float) -> float:
    """2^ceil(log2(amax / 127)), at least 2^-126; 1 for 0."""
    if amax == 0.0:
        return 1.0
    m, e = math.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 127 = 0.9921875 2^7
    return math.ldexp(1.0, max(-126, e - 7 if m <= 0.9921875 else e - 6))


def bounds_of(k):
    """(int8 [heads, 2, d], steps [heads]) of a block's keys [n, heads, d], in fp64."""
    n, heads, d = k.shape
    out, steps = torch.zeros(heads, 2, d, dtype=torch.int8), torch.zeros(heads)
    for h in range(heads):
        x = k[:, h]
        finite = x[torch.isfinite(x)]
        s = step_of(float(finite.abs().max()) if finite.numel() else 0.0)
        lo = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x).amin(0)
        hi = torch.where(torch.isnan(x), torch.full_like(x, math.inf), x).amax(0)
        out[h, 0] = torch.floor(lo / s).clamp(-127, 127).to(torch.int8)
        out[h, 1] = torch.ceil(hi / s).clamp(-127, 127).to(torch.int8)
        steps[h] = s
    return out, steps


def whole(q):
    """The group's query rows [g, d] (fp64) in whole steps."""
    finite = q[torch.isfinite(q)]
    s = step_of(float(finite.abs().max()) if finite.numel() else 0.0)
    return torch.round(torch.nan_to_num(q, nan=0.0, posinf=math.inf, neginf=-math.inf) / s).clamp(-127, 127)


def scores(q, bounds, steps):
    """q [g, d] in whole steps, bounds [n, 2, d], steps [n]: the blocks' scores (fp64, exact)."""
    b = bounds.double()
    x = torch.maximum(q[:, None] * b[None, :, 0], q[:, None] * b[None, :, 1]).sum(-1)  # [g, n]
    return x.amax(0) * steps.double()


def pick(score, n, nsel, first, local):
    """The ascending list of blocks among the first n."""
    if n <= nsel:
        return list(range(n))
    sure = set(range(first)) | set(range(n - local, n))
    rest = sorted((i for i in range(n) if i not in sure), key=lambda i: (-float(score[i]), i))
    return sorted(sure | set(rest[:nsel - len(sure)]))

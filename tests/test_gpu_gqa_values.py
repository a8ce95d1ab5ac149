"""Dense grouped-head attention, key by key: a value row that is skipped, read
twice, or read from another key's place shows, however many keys there are.

The values are indicators: dim d of head h is not 0 at one key only, so that
out[t][h'][d] is that key's weight (times its scale) and has to be right to a
few half steps of itself; a key behind the query's position gives 0.  In
rounds over the keys every key is the one."""

from __future__ import annotations

import pytest
import torch

import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R
from test_gpu_gqa import CALLS, DEV, Case

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24

KEYS = {
    # (contexts, new tokens, hq, hkv, d, e4m3, page), (rounds or 0: every key)
    "one": (([5000], [1], 16, 8, 128, False, 64), 0),
    "one e4m3": (([5000], [1], 16, 8, 128, True, 64), 0),
    "long": (([150001], [1], 64, 8, 128, False, 16), 25),
    "long e4m3": (([150001], [1], 64, 8, 128, True, 64), 25),
    "long d64 e4m3": (([150001], [1], 32, 8, 64, True, 0), 25),
    "many": (([61 + 211 * i % 3000 for i in range(90)], [1] * 90, 32, 8, 64, False, 0), 0),
    "many e4m3": (([61 + 211 * i % 3000 for i in range(90)], [1] * 90, 32, 8, 128, True, 16), 0),
    "drafts": (([61 + 211 * i % 3000 for i in range(60)], [4] * 60, 64, 8, 128, False, 64), 0),
    "drafts e4m3": (([61 + 211 * i % 3000 for i in range(60)], [4] * 60, 64, 8, 128, True, 64), 0),
    "two tokens e4m3": (([9001, 300], [2, 2], 16, 2, 128, True, 64), 20),
    "prompt": (([2500], [2500], 8, 2, 128, False, 0), 0),
    "prompt d64": (([2500], [2500], 8, 4, 64, False, 0), 0),
    "packed": (([5, 300, 1, 131, 64, 777], [5, 300, 1, 131, 64, 777], 16, 2, 128, False, 0), 0),
    "chunk e4m3": (([3000, 1700, 90], [700, 64, 90], 16, 2, 128, True, 64), 0),
    "chunk e4m3 d64": (([3000, 1700, 90], [700, 64, 90], 16, 4, 64, True, 16), 0),
    "chunk pages of 16": (([3000, 1700, 90], [700, 64, 90], 16, 2, 128, False, 16), 0),
    "far": (([9000, 3100, 40], [9, 70, 40], 16, 2, 128, False, 64), 20),
    "far e4m3": (([9000, 3100, 40], [9, 70, 40], 16, 2, 128, True, 64), 20),
}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("name", list(KEYS))
def test_every_key_counts_once(name, call):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    (ctx, new, hq, hkv, d, e4m3, page), rounds = KEYS[name]
    c = Case(ctx, new, hq, hkv, d, e4m3=e4m3, page=page, seed=len(name))
    G, B = hq // hkv, len(ctx)
    rows = [R.rows_of(c.table, page, c.base, b, n).to(DEV) for b, n in enumerate(ctx)]
    q = c.dq.double()
    weights, tols = [], []
    for b, n in enumerate(ctx):
        k = R.values(c.dk[rows[b]], None if c.dks is None else c.dks[rows[b]])  # [n, hkv, d]
        qb = q[c.q_start[b]:c.q_start[b + 1]].view(new[b], hkv, G, d)
        s = torch.einsum("thgd,nhd->thgn", qb, k) * c.sm_scale
        mag = torch.einsum("thgd,nhd->thgn", qb.abs(), k.abs()).amax() * c.sm_scale
        pos = torch.tensor(c.pos[c.q_start[b]:c.q_start[b + 1]], device=DEV)
        hidden = torch.arange(n, device=DEV)[None] > pos[:, None]
        top_s = float(s.abs().max())
        s.masked_fill_(hidden[:, None, None, :], -torch.inf)
        weights.append(torch.softmax(s, -1).view(new[b], hq, n))
        score = EPS * (d * float(mag) + 8 * 1.4427 * 2 * top_s)
        # relative: half a step of the weight and of the result, the scores, the sum of the weights
        tols.append(2 * 2.0 ** -8 + 2.0 ** -16 + 2 * score + 2 * EPS * (n / 16 + 64))
        del s, k
    live = c.live.to(DEV)
    step = hkv * d
    every = (max(ctx) + step - 1) // step
    heads, dims = torch.arange(hkv, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    # spread over the keys when they are too many for all: the borders of tiles, pages, pieces come by
    for r in range(every) if not rounds or rounds >= every else [i * (every - 1) // (rounds - 1) for i in range(rounds)]:
        c.dv[live] = 0
        want = []
        for b, n in enumerate(ctx):
            key = (r * step + heads * d + dims) % n  # [hkv, d]
            c.dv[rows[b][key], heads, dims] = 0x38 if e4m3 else 1.0
            val = c.dvs[rows[b][key], heads].double() if e4m3 else torch.ones(hkv, d, dtype=torch.float64, device=DEV)
            w = weights[b].view(new[b], hkv, G, n)
            hit = torch.gather(w, 3, key[None, :, None, :].expand(new[b], hkv, G, d))
            want.append((hit * val[None, :, None, :]).view(new[b], hq, d))
        c.run(call)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        out = c.out.double()
        for b in range(B):
            err = (out[c.q_start[b]:c.q_start[b + 1]] - want[b]).abs()
            bad = err > tols[b] * want[b]
            assert not bool(bad.any()), f"round {r}, sequence {b}: {int(bad.sum())} weights, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ctx, new, hq, hkv, d", [([65536], [2048], 16, 2, 128), ([65536], [2048], 16, 2, 64),
                                                  ([26088, 26448], [360, 720], 16, 2, 128),
                                                  ([3000 + 17 * i for i in range(40)], [100 + i for i in range(40)], 8, 2, 128),
                                                  ([200 + 7 * i for i in range(150)], [3 + i % 50 for i in range(150)], 8, 2, 64)])
def test_prompts_give_the_same_bits_every_time(ctx, new, hq, hkv, d, e4m3):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    c = Case(ctx, new, hq, hkv, d, e4m3=e4m3, page=64, seed=3).run("prefill")
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(20):
        c.run("prefill")
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    assert int(c.status.item()) == 0

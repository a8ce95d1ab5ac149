"""Dense grouped-head attention where the cache ends: rows and pages outside it
count as zeros, are reported where a query sees them, and change nothing for
the queries that do not."""

from __future__ import annotations

import math

import pytest
import torch

import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R
from test_gpu_gqa import CALLS, DEV, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


def _check(c, b, tokens, k=None, v=None):
    """Rows `tokens` of sequence b against the 64-bit form (over k, v: its keys and values)."""
    torch.cuda.synchronize()
    rows = R.rows_of(c.table, c.page, c.base, b, c.ctx[b])
    if k is None:
        k, v = R.values(c.k[rows], None if c.ks is None else c.ks[rows]), R.values(c.v[rows], None if c.vs is None else c.vs[rows])
    idx = torch.tensor([c.q_start[b] + t for t in tokens])
    pos = [c.pos[int(i)] for i in idx]
    ref, rl, tol, ltol = R.attend(c.q[idx].double(), k, v, pos, c.sm_scale)
    assert bool(((c.out.double().cpu()[idx] - ref).abs() <= tol).all())
    assert bool(((c.lse.double().cpu()[idx] - rl).abs() <= ltol).all())


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ctx, inside", [(130, 129), (130, 70), (70, 65), (1000, 930), (3000, 2990)])
def test_contexts_that_run_past_the_cache(call, e4m3, ctx, inside):
    """ctx_len counts rows past the cache: queries that stay inside are served, silently; one that sees a
    row outside reports it, and that row counts as zeros."""
    pos = [3, inside - 1, inside // 2]
    c = Case([ctx], [3], 16, 2, 128, e4m3=e4m3, pos=pos)
    c.seqs.num_rows = c.base[0] + inside
    c.run(call).check()
    c.pos[0] = ctx - 1
    c.d_pos[0] = ctx - 1
    c.run(call)
    assert int(c.status.item()) == 6
    _check(c, 0, [1, 2])
    rows = R.rows_of(None, 0, c.base, 0, ctx)
    k, v = [R.values(x[rows], None if s is None else s[rows]) for x, s in ((c.k, c.ks), (c.v, c.vs))]
    k[inside:], v[inside:] = 0, 0
    _check(c, 0, [0], k, v)


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_a_last_page_partly_inside(call, e4m3, page):
    ctx, inside = 5 * page, 4 * page + page // 2 + 1
    c = Case([ctx], [3], 8, 2, 128, e4m3=e4m3, page=page, pos=[inside - 1, 0, 4 * page], spare=0, dirty=False)
    c.table[0] = torch.arange(5, dtype=torch.int32)
    c.seqs.page_table.copy_(c.table)
    c.seqs.num_rows = inside
    c.run(call).check()
    c.d_pos[1] = c.pos[1] = inside
    c.run(call)
    assert int(c.status.item()) == 6
    _check(c, 0, [0, 2])


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_page_leaves_the_queries_before_it(call, e4m3, bad):
    """Sequences with a bad page between sequences of values that are not finite: the queries before the page
    are served, those behind it see zeros there."""
    B = 400
    c = Case([700] * B, [2] * B, 16, 2, 128, e4m3=e4m3, page=64, pos=[300, 690] * B)
    for b in range(0, B, 2):
        rows = R.rows_of(c.table, 64, None, b, 700)
        c.dv[rows] = 0x7F if e4m3 else math.inf
        c.dk[rows[::3]] = 0x7F if e4m3 else math.nan
        if e4m3:
            c.dvs[rows[::5]] = math.nan
            c.dks[rows[::7]] = math.inf
    c.seqs.page_table[1::2, 5] = bad
    c.run(call)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 6
    for b in range(1, B, 2):
        _check(c, b, [0])
    for b in (1, B // 2 + 1, B - 1):
        rows = R.rows_of(c.table, 64, None, b, 700)
        k, v = [R.values(x[rows], None if s is None else s[rows]) for x, s in ((c.k, c.ks), (c.v, c.vs))]
        k[320:384], v[320:384] = 0, 0
        _check(c, b, [1], k, v)

"""Dense grouped-head attention on a GB300 through the C ABI: K/V cache writes
with the rotation, decode and prompts, against the 64-bit forms and error
bounds of gqa_reference.py."""

from __future__ import annotations

import math

import pytest
import torch

import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = {"decode": dsa.dense_gqa_decode, "prefill": dsa.dense_gqa_prefill}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


class Case:
    """Sequences over random caches (every unused row NaN), and their results."""

    def __init__(self, ctx, new, hq, hkv, d, *, e4m3=False, page=0, pos=None, seed=0, stride=None, one_buffer=False,
                 spare=3, dirty=True, extra_q=0, amp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.hq, self.hkv, self.d, self.e4m3, self.page = ctx, new, hq, hkv, d, e4m3, page
        B = len(ctx)
        self.q_start = [0]
        for m in new:
            self.q_start.append(self.q_start[-1] + m)
        self.nq = self.q_start[-1]
        self.pos = pos if pos is not None else [n - m + i for n, m in zip(ctx, new) for i in range(m)]
        if page:
            used = [(n + page - 1) // page for n in ctx]
            order = torch.randperm(sum(used) + spare, generator=g)
            self.table = torch.zeros(B, max(1, max(used)), dtype=torch.int32)
            at = 0
            for b, u in enumerate(used):
                self.table[b, :u] = order[at:at + u].int()
                at += u
            self.rows, self.base = (sum(used) + spare) * page, None
        else:
            self.table = None
            self.base = [spare + sum(ctx[:b]) + 2 * b for b in range(B)]
            self.rows = self.base[-1] + ctx[-1] + spare
        self.live = torch.zeros(self.rows, dtype=torch.bool)
        for b, n in enumerate(ctx):
            self.live[R.rows_of(self.table, page, self.base, b, n)] = True
        self.q = (torch.randn(self.nq + extra_q, hq, d, generator=g) * amp).bfloat16()
        if e4m3:
            shape = (self.rows, hkv, d)
            self.k, self.v = [(torch.randn(shape, generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
                              .view(torch.uint8) for _ in range(2)]
            self.ks, self.vs = [torch.rand(self.rows, hkv, generator=g) * 0.01 + 0.002 for _ in range(2)]
            if dirty:
                for t in (self.k, self.v):
                    t[~self.live] = 0x7F
                for t in (self.ks, self.vs):
                    t[~self.live] = math.nan
        else:
            self.k, self.v = [torch.randn(self.rows, hkv, d, generator=g).bfloat16() for _ in range(2)]
            self.ks = self.vs = None
            if dirty:
                self.k[~self.live] = math.nan
                self.v[~self.live] = math.inf
        self.sm_scale = 1.0 / math.sqrt(d)
        dt = dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16
        if one_buffer:  # K and V of a row beside each other, and a gap behind them
            buf = torch.zeros(self.rows, 2 * hkv + 1, d, dtype=self.k.dtype, device=DEV)
            self.dk, self.dv = buf[:, :hkv], buf[:, hkv:2 * hkv]
            self.dk.copy_(self.k)
            self.dv.copy_(self.v)
            qbuf = torch.zeros(self.q.shape[0], hq + 1, d, dtype=torch.bfloat16, device=DEV)
            self.dq = qbuf[:, :hq]
            self.dq.copy_(self.q)
        else:
            self.dk, self.dv, self.dq = self.k.to(DEV), self.v.to(DEV), self.q.to(DEV)
        self.shape = dsa.GqaShape(hq, hkv, d, dt, q_stride=self.dq.stride(0), k_stride=self.dk.stride(0),
                                  v_stride=self.dv.stride(0))
        self.dks = None if self.ks is None else self.ks.to(DEV)
        self.dvs = None if self.vs is None else self.vs.to(DEV)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.d_pos = torch.tensor(self.pos + [0] * extra_q, **i32)
        self.d_start = torch.tensor(self.q_start, **i32)
        self.d_ctx = torch.tensor(ctx, **i32)
        self.seqs = dsa.Seqs(self.d_ctx, self.d_start, self.d_pos, max_ctx=max(1, max(ctx)),
                             max_q_per_seq=max(1, max(new)), num_rows=self.rows,
                             page_table=None if self.table is None else self.table.to(DEV), page_size=page,
                             seq_base=None if self.base is None else
                             torch.tensor(self.base, dtype=torch.int64, device=DEV))
        self.num_q = self.nq + extra_q
        n = dsa.dense_gqa_workspace_size(self.shape, self.seqs, self.num_q)
        # a workspace full of NaN: nothing of it may be read before it is written
        self.ws = torch.full((max(1, n) // 4 + 64,), math.nan, dtype=torch.float32, device=DEV).view(torch.uint8)
        self.ws_bytes = n

    def run(self, call, stream=None, lse=True):
        self.out = torch.full((self.num_q, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.num_q, self.hq), 7.0, dtype=torch.float32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.again(call, stream, lse)
        return self

    def again(self, call, stream=None, lse=True):
        CALLS[call](self.shape, self.dq, self.dk, self.dv, self.dks, self.dvs, self.seqs, self.num_q, self.sm_scale,
                    self.out, self.lse if lse else None, self.ws, self.ws_bytes, d_status=self.status, stream=stream)

    def check(self, seqs=None, status=0, max_rows=24):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        k, v = R.values(self.k, self.ks), R.values(self.v, self.vs)
        for b in range(len(self.ctx)) if seqs is None else seqs:
            rows = R.rows_of(self.table, self.page, self.base, b, self.ctx[b])
            m = self.new[b]
            pick = range(m) if m <= max_rows else sorted({0, 1, m - 2, m - 1} | {i * m // 16 for i in range(16)})
            idx = torch.tensor([self.q_start[b] + i for i in pick], dtype=torch.long)
            pos = [self.pos[int(i)] for i in idx]
            ref, rl, tol, ltol = R.attend(self.q[idx].double(), k[rows], v[rows], pos, self.sm_scale)
            err = (out[idx] - ref).abs()
            assert bool((err <= tol).all()), f"sequence {b}: off by {float((err - tol).max()):.3g} more than allowed"
            for i, p in enumerate(pos):
                if p < 0:
                    assert bool((lse[idx[i]] == -math.inf).all())
                else:
                    e = (lse[idx[i]] - rl[i]).abs()
                    assert bool((e <= ltol[i]).all()), f"sequence {b}: lse off by {float((e - ltol[i]).max()):.3g}"


DECODE = {
    # (contexts, new tokens, hq, hkv, d, e4m3, page)
    "one token": ([1], [1], 8, 1, 128, False, 0),
    "two lengths": ([63, 64, 65], [1, 1, 1], 8, 2, 128, False, 64),
    "long": ([9001], [1], 16, 2, 128, False, 64),
    "long e4m3": ([9001], [1], 16, 2, 128, True, 64),
    "pages of 16": ([130, 17, 1, 300], [1, 1, 1, 1], 8, 2, 128, False, 16),
    "pages of 16 e4m3": ([130, 17, 1, 300], [1, 1, 1, 1], 8, 2, 128, True, 16),
    "pages of 32 d64": ([130, 33, 1, 300], [1, 1, 1, 1], 4, 4, 64, False, 32),
    "pages of 256 d64 e4m3": ([513, 33, 1, 300], [1, 1, 1, 1], 6, 3, 64, True, 256),
    "pages of 16 d64 e4m3": ([513, 33, 1, 300], [1, 2, 1, 1], 6, 3, 64, True, 16),
    "odd group": ([200, 777], [1, 1], 14, 2, 128, False, 64),
    "group of 12": ([200, 777], [1, 1], 12, 1, 64, False, 0),
    "verify": ([200, 777, 6], [4, 1, 5], 16, 2, 128, False, 64),
    "verify e4m3": ([200, 777, 6, 64], [4, 1, 5, 4], 16, 2, 128, True, 64),
    "verify d64": ([200, 777, 6, 64], [4, 1, 5, 4], 14, 2, 64, False, 64),
    "group of 64": ([300, 64], [2, 1], 64, 1, 128, False, 64),
    "many sequences": ([1 + 37 * i % 400 for i in range(130)], [1] * 130, 4, 2, 64, False, 64),
    "more heads than lanes": ([70, 300], [1, 1], 40, 40, 64, False, 64),
    "empty among them": ([0, 90, 0, 5], [0, 1, 0, 1], 8, 2, 128, False, 64),
}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("name", list(DECODE))
def test_few_tokens(name, call):
    ctx, new, hq, hkv, d, e4m3, page = DECODE[name]
    Case(ctx, new, hq, hkv, d, e4m3=e4m3, page=page, seed=len(name)).run(call).check()


PROMPTS = {
    "one token": ([1], [1], 8, 1, 128, False, 0),
    "tile": ([128], [128], 8, 2, 128, False, 0),
    "tile and one": ([129], [129], 8, 2, 128, False, 0),
    "packed": ([5, 300, 1, 131, 64], [5, 300, 1, 131, 64], 16, 2, 128, False, 0),
    "packed d64": ([5, 300, 1, 131, 64], [5, 300, 1, 131, 64], 16, 4, 64, False, 0),
    "ungrouped": ([5, 300, 257], [5, 300, 257], 3, 3, 128, False, 0),
    "group of 64": ([70, 9], [70, 9], 64, 1, 64, False, 0),
    "odd group": ([5, 300, 257], [5, 300, 257], 14, 2, 128, False, 0),
    "chunk": ([700, 1000, 90], [200, 64, 90], 16, 2, 128, False, 64),
    "chunk pages of 16": ([700, 1000, 90], [200, 64, 90], 16, 2, 128, False, 16),
    "chunk pages of 256": ([700, 1000, 90], [200, 64, 90], 8, 1, 64, False, 256),
    "chunk e4m3": ([700, 1000, 90], [200, 64, 90], 16, 2, 128, True, 64),
    "chunk e4m3 d64": ([700, 1000, 90], [200, 64, 90], 10, 2, 64, True, 16),
    "no tokens among them": ([40, 90, 0, 5], [0, 90, 0, 3], 8, 2, 128, False, 64),
    "long": ([2500], [2500], 8, 2, 128, False, 0),
    # few tokens far into their sequences: the keys are split and joined
    "many": ([1 + 53 * i % 211 for i in range(150)], [1 + 53 * i % 211 for i in range(150)], 8, 2, 64, False, 0),
    "many chunks": ([40 + 97 * i % 500 for i in range(170)], [i % 40 for i in range(170)], 4, 1, 128, False, 16),
    "far": ([5000, 3100, 40], [9, 70, 40], 16, 2, 128, False, 64),
    "far d64 pages of 16": ([5000, 3100, 1], [9, 70, 1], 12, 4, 64, False, 16),
    "far e4m3": ([5000, 3100, 40], [9, 70, 40], 16, 2, 128, True, 64),
    "far e4m3 d64": ([5000, 3100, 40], [9, 70, 40], 6, 1, 64, True, 32),
    "far ungrouped": ([4100], [300], 2, 2, 128, False, 0),
}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts(name, call):
    ctx, new, hq, hkv, d, e4m3, page = PROMPTS[name]
    Case(ctx, new, hq, hkv, d, e4m3=e4m3, page=page, seed=len(name)).run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [0, 64])
def test_keys_and_values_side_by_side(call, e4m3, page):
    """K and V in one buffer with a gap behind each row, q rows with a gap."""
    Case([200, 77], [3, 77], 8, 2, 128, e4m3=e4m3, page=page, one_buffer=True).run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_see_nothing_and_any_positions(call, e4m3):
    """Positions in no order, some -1 (no key): zeros and -inf; keys past every position are never used."""
    ctx, new = [150, 300, 0, 20], [5, 4, 2, 1]
    pos = [-1, 0, 149, -1, 3, 7, 7, 128, 63, -1, -1, -1]
    c = Case(ctx, new, 8, 2, 128, e4m3=e4m3, page=64, pos=pos)
    # sequence 1's keys past 128 are seen by none of its queries: whatever they hold
    rows = R.rows_of(c.table, 64, None, 1, 300)[129:]
    if e4m3:
        c.dv[rows] = 0x7F
        c.dvs[rows] = math.inf
    else:
        c.dv[rows] = math.nan
        c.dk[rows] = math.inf
    c.run(call).check()
    out = c.out.cpu()
    for i, p in enumerate(pos):
        if p < 0:
            assert bool((out[i] == 0).all())


@pytest.mark.parametrize("call", list(CALLS))
def test_rows_behind_the_last_sequence_stay(call):
    c = Case([90, 30], [3, 2], 8, 2, 128, page=64, extra_q=4).run(call)
    c.check()
    assert bool((c.out[c.nq:] == 7).all()) and bool((c.lse[c.nq:] == 7).all())


@pytest.mark.parametrize("call", list(CALLS))
def test_bad_positions_and_sequences_are_reported_and_skipped(call):
    c = Case([90, 30, 40], [3, 2, 1], 8, 2, 128, page=64)
    c.d_pos[1] = 90       # outside its context
    c.d_pos[3] = -2
    c.run(call)
    keep = c.new
    c.new = [1, 0, 1]
    c.check(seqs=[0, 2], status=6)
    c.new = keep
    assert bool((c.out[[1, 3]] == 7).all()) and bool((c.lse[[1, 3]] == 7).all())
    c = Case([90, 30, 40], [3, 2, 1], 8, 2, 128, page=64)
    c.d_ctx[1] = 91       # more than max_ctx
    c.run(call)
    c.check(seqs=[0, 2], status=6)
    assert bool((c.out[3:5] == 7).all()) and bool((c.lse[3:5] == 7).all())


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
def test_joined_rows_that_see_little_and_bad_ones(call, e4m3):
    """Where a row's keys are split: rows that see no key, one key, the keys of the first part only;
    a bad position and rows behind the last sequence stay unwritten; stale rows are not used."""
    pos = [-1, 0, 300, 2000, 5999, 64, 127, 128]
    c = Case([6000, 30], [8, 1], 8, 2, 128, e4m3=e4m3, page=64, pos=pos + [29], extra_q=3)
    c.run(call).check()
    assert bool((c.out[0] == 0).all()) and bool((c.out[c.nq:] == 7).all()) and bool((c.lse[c.nq:] == 7).all())
    c.d_pos[4] = 6000
    c.run(call)
    c.new[0] = 4
    c.check(status=6)
    assert bool((c.out[4] == 7).all()) and bool((c.lse[4] == 7).all())


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_pages_are_reported_and_not_read(call, bad):
    c = Case([90, 300, 40], [3, 2, 1], 8, 2, 128, page=64)
    c.seqs.page_table[1, 2] = bad
    c.run(call)
    c.check(seqs=[0, 2], status=6)


@pytest.mark.parametrize("call", list(CALLS))
def test_rows_outside_the_cache_are_reported_and_not_read(call):
    c = Case([90, 300, 40], [3, 2, 1], 8, 2, 128)
    c.seqs.seq_base[1] = c.rows - 299
    c.run(call)
    c.check(seqs=[0, 2], status=6)
    c = Case([90, 300, 40], [3, 2, 1], 8, 2, 128)
    c.seqs.seq_base[0] = -1
    c.run(call)
    c.check(seqs=[1, 2], status=6)


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("many", [False, True])
def test_rows_that_see_nothing_beside_values_that_are_not_finite(call, e4m3, many):
    """A row without keys is zeros and -inf, whatever the other rows of its sequence see; so are the
    sequences beside it what they are."""
    B = 45 if many else 2
    ctx, new = [3000] + [70] * (B - 1), [8] + [1] * (B - 1)
    pos = [-1, 2999, 40, -1, 2000, -1, -1, 64] + [69] * (B - 1)
    c = Case(ctx, new, 32, 8, 128, e4m3=e4m3, page=64, pos=pos)
    rows = R.rows_of(c.table, 64, None, 0, 3000)
    for j in (5, 1999, 2990):
        if e4m3:
            c.dv[rows[j]] = 0x7F
        else:
            c.dv[rows[j]] = math.nan if j == 5 else math.inf
    c.run(call).check(seqs=range(1, B))
    out, lse = c.out.cpu(), c.lse.cpu()
    for i in (0, 3, 5, 6):
        assert bool((out[i] == 0).all()) and bool((lse[i] == -math.inf).all())


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("where", ["first", "last", "many"])
def test_value_scales_far_apart(call, where):
    """e4m3: rows of zeros with a scale 2^20 times the others', and scales that grow along the sequence:
    a weight times its scale keeps 11 bits down to 2^-21 of the largest such product."""
    c = Case([700, 130], [3, 130], 16, 2, 128, e4m3=True, page=64)
    for b in range(2):
        rows = R.rows_of(c.table, 64, None, b, c.ctx[b])
        n = len(rows)
        c.vs[rows] *= 2.0 ** -20
        if where == "many":
            c.vs[rows] *= (2.0 ** (20 * torch.arange(n) // n).float())[:, None]
        else:
            at = rows[:2] if where == "first" else rows[n // 2:n // 2 + 2]
            c.v[at] = 0
            c.vs[at] = 1.0
    c.dv, c.dvs = c.v.to(DEV), c.vs.to(DEV)
    c.run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
def test_large_scores(call):
    """Scores of hundreds: one key takes all the weight, the reference moves often."""
    Case([700, 90], [2, 90], 8, 2, 128, page=64, amp=60.0).run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
def test_without_lse_and_other_scales(call):
    c = Case([300, 90], [2, 90], 8, 2, 128, page=64)
    c.run(call).check()
    want = c.out.clone()
    c.run(call, lse=False)
    torch.cuda.synchronize()
    assert torch.equal(want, c.out) and bool((c.lse == 7).all())
    for scale in (0.0, -0.3, 1e-9):
        c.sm_scale = scale
        c.run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
def test_same_bits_in_any_workspace_stream_or_graph(call, e4m3):
    c = Case([700, 90, 1500], [4, 90, 1], 16, 2, 128, e4m3=e4m3, page=64).run(call)
    c.check()
    want, wl = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.ws.zero_()
    side.wait_stream(torch.cuda.current_stream())
    c.run(call, stream=side)
    torch.cuda.synchronize()
    # run() fills its outputs on the current stream: once more, in order
    c.again(call, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(want, c.out) and torch.equal(wl, c.lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.again(call)
    for _ in range(2):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.ws.view(torch.float32).fill_(math.nan)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, c.out) and torch.equal(wl, c.lse)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("b, ctx, new, d", [(1, 262144, 1, 128), (40, 6000, 1, 128), (40, 6000, 2, 128), (1, 262144, 2, 64),
                                            (40, 6000, 4, 128), (6, 6000, 1, 128)])
def test_same_bits_whenever_the_loads_are_waited_for(b, ctx, new, d, e4m3):
    """Long caches, bound by memory: the same results every time, and those of the formula."""
    hq, hkv, rows = 64, 8, b * ctx
    g = torch.Generator(device=DEV).manual_seed(7)
    if e4m3:
        k, v = [torch.randint(0, 0x7F, (rows, hkv, d), generator=g, device=DEV, dtype=torch.uint8)
                | (torch.randint(0, 2, (rows, hkv, d), generator=g, device=DEV, dtype=torch.uint8) << 7) for _ in range(2)]
        ks, vs = [torch.rand(rows, hkv, generator=g, device=DEV) * 0.004 + 0.004 for _ in range(2)]
    else:
        k, v = [torch.randn(rows, hkv, d, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
        ks = vs = None
    q = torch.randn(b * new, hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    pos = torch.arange(ctx - new, ctx, **i32).repeat(b)
    seqs = dsa.Seqs(torch.full((b,), ctx, **i32), torch.arange(0, b * new + 1, new, **i32), pos, max_ctx=ctx,
                    max_q_per_seq=new, num_rows=rows,
                    seq_base=torch.arange(0, rows, ctx, dtype=torch.int64, device=DEV))
    shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16)
    nb = dsa.dense_gqa_workspace_size(shape, seqs, b * new)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, **i32)
    scale = 1 / math.sqrt(d)

    def run():
        out = torch.empty_like(q)
        lse = torch.empty(b * new, hq, device=DEV)
        dsa.dense_gqa_decode(shape, q, k, v, ks, vs, seqs, b * new, scale, out, lse, ws, nb, d_status=status)
        return out, lse

    out, lse = run()
    for _ in range(20):
        o, l = run()
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert int(status.item()) == 0
    s, h = b - 1, 3  # one sequence's heads of one key head
    kk = R.values(k[s * ctx:, h:h + 1], None if ks is None else ks[s * ctx:, h:h + 1])[:, 0]
    vv = R.values(v[s * ctx:, h:h + 1], None if vs is None else vs[s * ctx:, h:h + 1])[:, 0]
    for t in range(new):
        n = ctx - new + t + 1
        p = torch.softmax(scale * (kk[:n] @ q[s * new + t, h * 8:h * 8 + 8].double().T), 0)
        ref, av = p.T @ vv[:n], p.T @ vv[:n].abs()
        # a half step of the result; weights off by a half step each, in no one direction: a
        # twentieth of the worst case; sums of n / 16 fp32 additions
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 / 20 + 2.0 ** -24 * (n / 16 + 64) * 2) * av
        assert bool(((out[s * new + t, h * 8:h * 8 + 8].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("call", list(CALLS))
def test_two_calls_at_once(call):
    """Two streams, a workspace each."""
    a = Case([3000, 90], [1, 90], 16, 2, 128, page=64, seed=1).run(call)
    b = Case([2000, 900], [2, 9], 16, 2, 128, page=64, seed=2).run(call)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.again(call, s1)
        b.again(call, s2)
    a.check()
    b.check()


@pytest.mark.parametrize("call", list(CALLS))
def test_offsets_past_32_bits(call):
    """Rows 2^16 elements apart: the last ones lie past 2^32 elements."""
    rows, wide = 66000, 65536
    buf = torch.empty(rows, wide, dtype=torch.bfloat16, device=DEV)
    c = Case([200], [3], 8, 2, 128)
    for x, off in ((c.k, 0), (c.v, 1024)):
        buf[rows - 200:, off:off + 256] = x[c.base[0]:c.base[0] + 200].reshape(200, 256).to(DEV)
    c.dk, c.dv = buf, buf[:, 1024:]
    c.shape = dsa.GqaShape(8, 2, 128, dsa.DSA_BF16, k_stride=wide, v_stride=wide)
    c.seqs.num_rows = rows
    c.seqs.seq_base[0] = rows - 200
    c.run(call).check()


# ---------------------------------------------------------------------------
# cache writes
INSERTS = {
    # n, hq, hkv, d, e4m3, rot, halves
    "one token": (1, 8, 2, 128, False, 64, False),
    "halves": (37, 8, 2, 128, False, 128, True),
    "part of the halves": (37, 6, 3, 128, False, 48, True),
    "pairs": (300, 5, 5, 128, False, 128, False),
    "no rotation": (65, 8, 2, 128, False, 0, False),
    "no queries": (65, 0, 2, 64, False, 64, True),
    "d64": (130, 12, 4, 64, False, 32, True),
    "e4m3": (130, 16, 2, 128, True, 64, False),
    "e4m3 halves": (130, 0, 8, 128, True, 128, True),
    "e4m3 d64": (65, 3, 1, 64, True, 16, False),
    "many": (2500, 16, 2, 128, False, 64, True),
}


def _half_step(exact, q):
    """Half a step of a format with q bits behind the leading one (normal values), for exact values."""
    a = exact.abs().clamp(min=2.0 ** -126)
    return torch.exp2(torch.floor(torch.log2(a)) - q) / 2


def _check_rows(got, exact, what):
    """bf16 rows: the nearest value, up to the fp32 evaluation (two products and a sum of values
    up to the pair's size, a cosine and sine off by 3e-7: 2e-6 of the row's largest is above them)."""
    err = (got.double() - exact).abs()
    slack = 2e-6 * exact.abs().amax(-1, keepdim=True)
    bad = err > _half_step(exact, 7) * (1 + 1e-9) + slack
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values are not the nearest"


def _check_codes(codes, scale, exact, what):
    want, ws = R.quantise(exact)
    assert bool(((scale.double() - ws).abs() <= 3e-6 * ws).all()), f"{what}: scale"
    got = codes.view(torch.float8_e4m3fn).double()
    # half a step of e4m3 (3 bits; 2^-10 below 2^-6), and the scale's and rotation's fp32 slack
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -6))) - 3) / 2
    bad = (got - want).abs() > step * (1 + 1e-9) + 3e-6 * 448
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes are not the nearest"


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("name", list(INSERTS))
def test_insert(name, fused):
    n, hq, hkv, d, e4m3, rot, halves = INSERTS[name]
    g = torch.Generator().manual_seed(n + d)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    pos[0] = 0
    rows = 2 * n + 5
    slot = torch.randperm(rows, generator=g)[:n]
    skip = torch.zeros(n, dtype=torch.bool)
    if n > 4:
        skip[n // 2] = True
        slot[n // 2] = -1
    if fused:
        x = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16()
        dx = x.to(DEV)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        dq, dk, dv = dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:]
    else:
        q, k, v = [torch.randn(n, h, d, generator=g).bfloat16() for h in (hq, hkv, hkv)]
        dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    inv = (10000.0 ** (-torch.arange(0, rot, 2).double() / max(1, rot))).float() if rot else None
    # K and V rows in one buffer
    kind = torch.uint8 if e4m3 else torch.bfloat16
    buf = torch.full((rows, 2 * hkv, d), 9, dtype=kind, device=DEV)
    ks = torch.full((rows, hkv), 9.0, device=DEV) if e4m3 else None
    vs = torch.full((rows, hkv), 9.0, device=DEV) if e4m3 else None
    qo = torch.full((n, max(1, hq), d), 9.0, dtype=torch.bfloat16, device=DEV) if hq else None
    shape = dsa.GqaShape(max(hq, hkv), hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16,
                         k_stride=2 * hkv * d, v_stride=2 * hkv * d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.dsa_kv_insert(shape, dk, dv, dq if hq else None, pos.to(DEV), slot.to(DEV), n,
                      None if inv is None else inv.to(DEV), rot,
                      dsa.DSA_ROPE_HALVES if halves else dsa.DSA_ROPE_PAIRS, buf, buf[:, hkv:], ks, vs, rows, qo,
                      k_stride=dk.stride(0), v_stride=dv.stride(0), q_stride=dq.stride(0) if hq else 0,
                      d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rk = R.rotate(k.double(), pos, inv, rot, halves)
    b = buf.cpu()
    at = slot[~skip]
    if e4m3:
        _check_codes(b[at, :hkv], ks.cpu()[at], rk[~skip], "K")
        _check_codes(b[at, hkv:], vs.cpu()[at], v.double()[~skip], "V")
    else:
        _check_rows(b[at, :hkv], rk[~skip], "K")
        assert torch.equal(b[at, hkv:], v[~skip]), "V is copied"
    if hq:
        _check_rows(qo.cpu(), R.rotate(q.double(), pos, inv, rot, halves), "q")  # a skipped slot's too
    rest = torch.ones(rows, dtype=torch.bool)
    rest[at] = False
    assert bool((b[rest] == 9).all())
    if e4m3:
        assert bool((ks.cpu()[rest] == 9).all()) and bool((vs.cpu()[rest] == 9).all())


def test_insert_reports_and_skips_bad_tokens():
    n, hq, hkv, d = 6, 4, 2, 128
    g = torch.Generator().manual_seed(3)
    q, k, v = [torch.randn(n, h, d, generator=g).bfloat16() for h in (hq, hkv, hkv)]
    pos = torch.tensor([5, -1, 7, -1, 9, 4], dtype=torch.int32)
    slot = torch.tensor([3, 4, 20, -1, -7, 0])
    bufk, bufv = [torch.full((20, hkv, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    qo = torch.full((n, hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    inv = torch.rand(32, generator=g)
    shape = dsa.GqaShape(hq, hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.dsa_kv_insert(shape, k.to(DEV), v.to(DEV), q.to(DEV), pos.to(DEV), slot.to(DEV), n, inv.to(DEV), 64,
                      dsa.DSA_ROPE_PAIRS, bufk, bufv, None, None, 20, qo, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 6
    rk = R.rotate(k.double(), pos, inv, 64, False)
    rq = R.rotate(q.double(), pos, inv, 64, False)
    for i, s in ((0, 3), (5, 0)):
        _check_rows(bufk[s].cpu()[None], rk[i][None], "K")
        assert torch.equal(bufv[s].cpu(), v[i])
    rest = [r for r in range(20) if r not in (0, 3)]
    assert bool((bufk[rest] == 9).all()) and bool((bufv[rest] == 9).all())
    for i in (0, 4, 5):
        _check_rows(qo[i].cpu()[None], rq[i][None], "q")
    assert bool((qo[[1, 2, 3]] == 9).all())


@pytest.mark.parametrize("halves", [False, True])
def test_insert_rotates_queries_in_place(halves):
    n, hq, hkv, d = 50, 8, 2, 128
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16()
    dx = x.to(DEV)
    pos = torch.arange(n, dtype=torch.int32)
    inv = torch.rand(64, generator=g)
    k_cache, v_cache = [torch.zeros(n, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    shape = dsa.GqaShape(hq, hkv, d, q_stride=dx.stride(0))
    dsa.dsa_kv_insert(shape, dx[:, hq:], dx[:, hq + hkv:], dx, pos.to(DEV), torch.arange(n, device=DEV), n,
                      inv.to(DEV), 128, dsa.DSA_ROPE_HALVES if halves else dsa.DSA_ROPE_PAIRS, k_cache, v_cache, None,
                      None, n, dx, k_stride=dx.stride(0), v_stride=dx.stride(0), q_stride=dx.stride(0))
    torch.cuda.synchronize()
    _check_rows(dx[:, :hq].cpu(), R.rotate(x[:, :hq].double(), pos, inv, 128, halves), "q")
    assert torch.equal(dx[:, hq:].cpu(), x[:, hq:])
    _check_rows(k_cache.cpu(), R.rotate(x[:, hq:hq + hkv].double(), pos, inv, 128, halves), "K")


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_then_tokens(e4m3):
    """The three calls as a server makes them: prompts written and attended to in two chunks, then
    three tokens one at a time, every result against the 64-bit attention over what the caches hold,
    and the caches against the 64-bit rotation."""
    hq, hkv, d, page = 16, 2, 128, 16
    lens, steps = [70, 5, 133], 3
    B = len(lens)
    g = torch.Generator().manual_seed(11)
    width = hq + 2 * hkv
    total = [n + steps for n in lens]
    xs = [torch.randn(n, width, d, generator=g).bfloat16() for n in total]
    maxp = max((n + page - 1) // page for n in total)
    table = torch.randperm(B * maxp, generator=g).view(B, maxp).int()
    rows = B * maxp * page
    kind = torch.uint8 if e4m3 else torch.bfloat16
    kc, vc = [torch.full((rows, hkv, d), 0x7F if e4m3 else math.nan, dtype=kind, device=DEV) for _ in range(2)]
    ks, vs = [torch.full((rows, hkv), math.nan, device=DEV) if e4m3 else None for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, 64, 2).double() / 64)).float()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = 1.0 / math.sqrt(d)
    done = [0] * B
    plans = [[n // 2 for n in lens], [n - n // 2 for n in lens]] + [[1] * B] * steps
    for step, new in enumerate(plans):
        x = torch.cat([xs[b][done[b]:done[b] + new[b]] for b in range(B)]).to(DEV)
        n = x.shape[0]
        pos = torch.cat([torch.arange(done[b], done[b] + new[b]) for b in range(B)]).int()
        slot = torch.cat([R.rows_of(table, page, None, b, total[b])[done[b]:done[b] + new[b]] for b in range(B)])
        q = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16)
        dsa.dsa_kv_insert(shape, x[:, hq:], x[:, hq + hkv:], x, pos.to(DEV), slot.to(DEV), n, inv.to(DEV), 64,
                          dsa.DSA_ROPE_HALVES, kc, vc, ks, vs, rows, q, k_stride=x.stride(0), v_stride=x.stride(0),
                          q_stride=x.stride(0), d_status=status)
        done = [a + b for a, b in zip(done, new)]
        start = torch.tensor([0] + new).cumsum(0).int().to(DEV)
        seqs = dsa.Seqs(torch.tensor(done, dtype=torch.int32, device=DEV), start, pos.to(DEV), max_ctx=max(done),
                        max_q_per_seq=max(new), num_rows=rows, page_table=table.to(DEV), page_size=page)
        nb = dsa.dense_gqa_workspace_size(shape, seqs, n)
        ws = torch.empty(max(1, nb), dtype=torch.uint8, device=DEV)
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(n, hq, device=DEV)
        call = dsa.dense_gqa_prefill if max(new) > 1 else dsa.dense_gqa_decode
        call(shape, q, kc, vc, ks, vs, seqs, n, scale, out, lse, ws, nb, d_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        k = R.values(kc.cpu(), None if ks is None else ks.cpu())
        v = R.values(vc.cpu(), None if vs is None else vs.cpu())
        _check_rows(q.cpu(), R.rotate(x[:, :hq].cpu().double(), pos, inv, 64, True), "q")
        at = 0
        for b in range(B):
            r = R.rows_of(table, page, None, b, done[b])
            if not e4m3:
                rk = R.rotate(xs[b][:done[b], hq:hq + hkv].double(), torch.arange(done[b]).int(), inv, 64, True)
                _check_rows(k[r], rk, "K")
            m = new[b]
            ref, rl, tol, ltol = R.attend(q[at:at + m].cpu().double(), k[r], v[r], pos[at:at + m], scale)
            assert bool(((out[at:at + m].cpu().double() - ref).abs() <= tol).all()), (step, b)
            assert bool(((lse[at:at + m].cpu().double() - rl).abs() <= ltol).all()), (step, b)
            at += m

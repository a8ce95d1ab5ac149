"""The step's plan, the writes of 8-bit caches with a scale per block of tokens
and head, and dense attention over them, on a GB300 through the C ABI, against
the plain forms of block_reference.py and gqa_reference.py."""

from __future__ import annotations

import math

import pytest
import torch

import block_reference as BR
import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R
from test_gpu_gqa import CALLS, Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = dsa._binding.DSA_ERR_BAD_INPUT


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# the plan
def _plan(cached, new, page, free, rng, num_pages, table, num_q, stream=None):
    """Runs dsa_step_plan; returns its results as lists and the status."""
    B = len(cached)
    o = dict(ctx=_i32([77] * B), q_start=_i32([77] * (B + 1)), q_pos=_i32([77] * num_q),
             slot=torch.full((num_q,), 77, dtype=torch.int64, device=DEV), next=_i32([77, 77]), table=_i32(table))
    status = _i32([0])
    free_t = _i32(free) if free else torch.empty(0, dtype=torch.int32, device=DEV)
    dsa.dsa_step_plan(_i32(cached), _i32(new), B, free_t, _i32(rng), page, num_pages, o["table"], num_q, o["ctx"],
                      o["q_start"], o["q_pos"], o["slot"], o["next"], d_status=status, stream=stream)
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in o.items()}, int(status)


def _requests(B, past, new, page, seed, width, spare=3):
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, past + 1, (B,), generator=g).tolist()
    fresh = torch.randint(0, new + 1, (B,), generator=g).tolist()
    pages = torch.randperm(B * width + spare, generator=g).tolist()
    table = [[-7] * width for _ in range(B)]
    at = 0
    for b in range(B):
        for c in range(-(-cached[b] // page)):
            table[b][c] = pages[at]
            at += 1
    return cached, fresh, pages[at:], len(pages), table


@pytest.mark.parametrize("B, past, new, page, spare", [
    (1, 0, 1, 16, 0), (1, 100, 300, 64, 5), (3, 64, 64, 64, 1), (64, 4000, 1, 64, 0), (513, 90, 40, 16, 7),
    (2048, 40, 3, 32, 100), (2049, 70, 5, 16, 0), (5000, 33, 2, 16, 1), (7, 9, 5000, 128, 2000),
])
def test_plan(B, past, new, page, spare):
    width = (past + new + page - 1) // page + 2
    cached, fresh, free, num_pages, table = _requests(B, past, new, page, B, width)
    num_q = sum(fresh) + spare
    free = [1 << 30] * 2 + free  # two pages that were taken before
    ref, bad = BR.plan(cached, fresh, page, free, [2, len(free)], num_pages, [list(r) for r in table], num_q)
    got, status = _plan(cached, fresh, page, free, [2, len(free)], num_pages, table, num_q)
    assert not bad and status == 0
    assert got == ref


REFUSED = {
    "too few pages": dict(cached=[10, 60, 5, 16], new=[40, 70, 1, 16], free=[3, 8, 1, 5], rng=[0, 4], num_q=127),
    "none at all": dict(cached=[10, 16], new=[3, 1], free=[], rng=[0, 0], num_q=4),
    "a later request that needs none": dict(cached=[16, 3], new=[20, 2], free=[3], rng=[0, 1], num_q=22),
    "rows past the end": dict(cached=[1, 2, 3], new=[4, 5, 6], free=list(range(3, 9)), rng=[0, 6], num_q=8),
    "no rows at all": dict(cached=[1, 2], new=[4, 0], free=[4], rng=[0, 1], num_q=0),
    "negative lengths": dict(cached=[-3, 2, 4], new=[4, -5, 6], free=list(range(3, 9)), rng=[0, 6], num_q=12),
    "longer than the table": dict(cached=[90, 2], new=[40, 5], free=list(range(3, 12)), rng=[0, 9], num_q=45),
    "a range outside the list": dict(cached=[10, 2], new=[40, 5], free=[3, 4], rng=[0, 3], num_q=45),
    "a range turned around": dict(cached=[10, 2], new=[40, 5], free=[3, 4], rng=[2, 1], num_q=45),
    "pages outside the cache": dict(cached=[10, 2], new=[40, 20], free=[3, 99, -4, 6], rng=[0, 4], num_q=60),
    "huge lengths": dict(cached=[2 ** 31 - 1, 5], new=[2 ** 31 - 1, 2], free=[3], rng=[0, 1], num_q=9),
}


@pytest.mark.parametrize("name", REFUSED)
def test_plan_refuses_requests(name):
    c = REFUSED[name]
    table = [[b * 8 + i for i in range(8)] for b in range(len(c["cached"]))]
    if name == "pages outside the cache":
        table[1][0] = 4000
    args = (c["cached"], c["new"], 16, c["free"], c["rng"], 64)
    ref, bad = BR.plan(*args, [list(r) for r in table], c["num_q"])
    got, status = _plan(*args, table, c["num_q"])
    assert bad and status == BAD
    assert got == ref


@pytest.mark.parametrize("past, new", [(2 ** 31 - 10, 20), (2 ** 31 - 21, 20), (2 ** 30 - 5, 6), (2 ** 30 - 5, 5)])
def test_plan_stops_at_the_longest_context(past, new):
    page, table = 1 << 20, [list(range(2100)), list(range(2100))]
    args = ([past, 3], [new, 4], page, [2100], [0, 1], 2200)
    ref, bad = BR.plan(*args, [list(r) for r in table], new + 4)
    got, status = _plan(*args, table, new + 4)
    assert bad == (past + new > 2 ** 30) and status == (BAD if bad else 0)
    assert got == ref


# ---------------------------------------------------------------------------
# writes
class Cache:
    """Sequences over a block-scaled cache with older tokens, and what an insert makes of it."""

    def __init__(self, past, new, hq, hkv, d, sb, *, page=0, seed=0, spare=2, gap=0, extra_q=0, rot=0, half=False,
                 amp=1.0, fused=False):
        g = torch.Generator().manual_seed(seed)
        self.past, self.new, self.sb, self.page, self.hq, self.hkv, self.d = past, new, sb, page, hq, hkv, d
        B = len(past)
        ctx = [p + n for p, n in zip(past, new)]
        unit = page or sb
        used = [-(-x // unit) for x in ctx]
        order = torch.randperm(sum(used) + spare, generator=g)
        self.rows = (sum(used) + spare) * unit
        self.table = self.base = None
        if page:
            self.table = torch.full((B, max(used) + 1), -1, dtype=torch.int32)
            at = 0
            for b, u in enumerate(used):
                self.table[b, :u] = order[at:at + u].int()
                at += u
        else:
            self.base = [sum(used[:b]) * sb for b in range(B)]
        self.q_start = [0]
        for n in new:
            self.q_start.append(self.q_start[-1] + n)
        nq = self.q_start[-1]
        self.num_q = nq + extra_q
        self.pos = [p + i for p, n in zip(past, new) for i in range(n)]
        buf = (torch.randn(self.num_q, hq + 2 * hkv + gap, d, generator=g) * amp).bfloat16()
        self.q, self.k, self.v = [x.clone() for x in (buf[:, :hq], buf[:, hq:hq + hkv], buf[:, hq + hkv:hq + 2 * hkv])]
        self.code = [(torch.randn(self.rows, hkv, d, generator=g) * 130).clamp(-448, 448).to(torch.float8_e4m3fn)
                     .view(torch.uint8) for _ in range(2)]
        self.scale = [torch.exp2(torch.randint(-14, -4, (self.rows // sb, hkv), generator=g).float()) for _ in range(2)]
        self.rot, self.half = rot, half
        self.inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None
        self.fused = fused
        self.ctx = ctx

    def rows_of(self, b, n=None):
        return R.rows_of(self.table, self.page, self.base, b, self.ctx[b] if n is None else n)

    def run(self, stream=None, queries=True, status=0, pos=None, ctx=None, inplace=False, num_rows=None):
        self.d_code = [x.to(DEV) for x in self.code]
        self.d_scale = [x.to(DEV) for x in self.scale]
        if self.fused:
            x = torch.cat([self.q, self.k, self.v], 1).to(DEV)
            q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
        else:
            q, k, v = self.q.to(DEV), self.k.to(DEV), self.v.to(DEV)
        self.q_out = q if inplace else torch.full((self.num_q, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        pos = (self.pos if pos is None else pos) + [3] * (self.num_q - len(self.pos))
        self.shape = dsa.GqaShape(self.hq, self.hkv, self.d, dsa.DSA_FP8_E4M3_BLOCKSCALE, scale_block=self.sb,
                                  q_stride=self.q_out.stride(0))
        self.seqs = dsa.Seqs(_i32(ctx or self.ctx), _i32(self.q_start), _i32(pos), max_ctx=max(max(ctx or self.ctx), 1),
                             max_q_per_seq=max(1, max(self.new)), num_rows=num_rows or self.rows,
                             page_table=None if self.table is None else self.table.to(DEV), page_size=self.page,
                             seq_base=None if self.base is None else torch.tensor(self.base, device=DEV))
        self.status = _i32([0])
        inv = None if self.inv is None else self.inv.to(DEV)
        dsa.dsa_kv_block_insert(self.shape, k, v, q if queries else None, self.seqs, self.num_q, inv, self.rot,
                                dsa.DSA_ROPE_HALVES if self.half else dsa.DSA_ROPE_PAIRS, self.d_code[0],
                                self.d_code[1], self.d_scale[0], self.d_scale[1], self.q_out if queries else None,
                                k_stride=k.stride(0), v_stride=v.stride(0), q_stride=q.stride(0),
                                d_status=self.status, stream=stream)
        torch.cuda.synchronize()
        assert int(self.status) == status
        return self

    def expect(self, skip=()):
        """The plain form's codes, scales and queries (fp64, before their rounding)."""
        code, scale = [x.clone() for x in self.code], [x.clone() for x in self.scale]
        pos = torch.tensor(self.pos, dtype=torch.int64)
        nq = len(self.pos)
        k = R.rotate(self.k[:nq].double(), pos, self.inv, self.rot, self.half)
        for b in range(len(self.past)):
            if b in skip or not self.new[b]:
                continue
            part = slice(self.q_start[b], self.q_start[b + 1])
            for x, c, s in ((k, code[0], scale[0]), (self.v[:nq].double(), code[1], scale[1])):
                BR.insert(x[part], c, s, self.rows_of(b), self.past[b], self.sb)
        return code, scale, k, R.rotate(self.q[:nq].double(), pos, self.inv, self.rot, self.half)

    def check(self, skip=(), queries=True):
        code, scale, k, q = self.expect(skip)
        got, gs = [x.cpu() for x in self.d_code], [x.cpu() for x in self.d_scale]
        assert torch.equal(gs[0], scale[0]) and torch.equal(gs[1], scale[1])
        assert torch.equal(got[1], code[1])
        if not self.rot:
            assert torch.equal(got[0], code[0])
        else:
            # the new keys: their rotation is off by a few fp32 roundings of the pair's size (angles too:
            # 2^-21 of it), then half a step of e4m3 (2^-4 of the value, 2^-10 of the scale where subnormal)
            fresh = torch.zeros(self.rows, dtype=torch.bool)
            for b in range(len(self.past)):
                if b in skip or not self.new[b]:
                    continue
                rows = self.rows_of(b)[self.past[b]:]
                fresh[rows] = True
                part = slice(self.q_start[b], self.q_start[b + 1])
                sc = scale[0][rows // self.sb].double()[..., None]
                val = BR.value_of(got[0][rows]) * sc
                size = self.k[part].double().abs().amax(-1, keepdim=True)
                tol = 2.0 ** -4 * k[part].abs() + 2.0 ** -10 * sc + 2.0 ** -19 * size
                assert bool(((val - k[part]).abs() <= tol).all())
            assert torch.equal(got[0][~fresh], code[0][~fresh])
        out = self.q_out.cpu()
        if not queries:
            return
        rows = [t for b in range(len(self.past)) if b not in skip for t in range(self.q_start[b], self.q_start[b + 1])]
        size = self.q[rows].double().abs().amax(-1, keepdim=True)
        assert bool(((out[rows].double() - q[rows]).abs() <= 2.0 ** -8 * q[rows].abs() + 2.0 ** -19 * size).all())
        left = sorted(set(range(self.num_q)) - set(rows))
        assert bool((out[left] == 7.0).all())


INSERTS = {
    # (past, new, hq, hkv, d, scale block, page)
    "one token": ([0], [1], 8, 1, 128, 64, 64),
    "one more token": ([5], [1], 8, 2, 128, 64, 64),
    "a token that opens a block": ([64, 16, 127], [1, 1, 1], 8, 2, 128, 16, 64),
    "a step of many": ([3 * i for i in range(70)], [1] * 70, 14, 2, 128, 64, 64),
    "drafts": ([60, 61, 62, 63, 64], [4, 4, 5, 4, 1], 5, 5, 64, 64, 64),
    "a prompt": ([0], [333], 16, 2, 128, 64, 64),
    "a chunk": ([77], [300], 12, 4, 128, 128, 128),
    "blocks of 16": ([13], [140], 8, 8, 64, 16, 32),
    "blocks of 32": ([31, 1], [140, 33], 8, 2, 128, 32, 256),
    "contiguous": ([7, 0, 100], [60, 1, 130], 8, 2, 128, 64, 0),
    "no tokens for some": ([7, 9, 0, 100], [0, 3, 0, 1], 8, 2, 64, 32, 64),
    "ungrouped": ([10], [100], 33, 33, 64, 64, 64),
}


@pytest.mark.parametrize("rot, half", [(0, False), (16, False), (64, True), (64, False)])
@pytest.mark.parametrize("name", INSERTS)
def test_insert(name, rot, half):
    past, new, hq, hkv, d, sb, page = INSERTS[name]
    Cache(past, new, hq, hkv, d, sb, page=page, rot=rot, half=half, seed=len(name), extra_q=2).run().check()


def test_insert_all_dims_rotated_far_positions():
    for half in (False, True):
        c = Cache([0, 40], [70, 3], 8, 2, 128, 64, page=64, rot=128, half=half, seed=3, fused=True)
        c.run().check()


def test_more_sequences_than_a_chunk_of_the_scan():
    n = 2300
    c = Cache([i % 5 for i in range(n)], [1 + i % 3 for i in range(n)], 2, 1, 64, 16, page=16, seed=5)
    c.run().check()


def test_sequences_without_a_page_between_others():
    """Pieces that are given up after their rows are on their way, the next ones of the same CTA behind them."""
    n = 2600
    c = Cache([i % 5 for i in range(n)], [1 + i % 3 for i in range(n)], 8, 2, 128, 16, page=16, rot=64, half=True, seed=6)
    lost = set(range(1, n, 3)) | set(range(1216, 1500))
    table = c.table.clone()
    c.table[sorted(lost)] = -1
    c.run(status=BAD)
    c.table = table
    c.check(skip=lost)


@pytest.mark.parametrize("amp", [1e-30, 2.0 ** -50, 1e-3, 300.0, 1e30])
def test_scales_of_any_size(amp):
    """Blocks' scales grow or stay, whichever the older tokens' scale asks for."""
    Cache([20, 64, 3], [30, 10, 1], 8, 2, 128, 64, page=64, amp=amp, seed=7).run().check()


def test_borders_of_the_scale_and_zeros():
    """Maxima of 448 2^k take 2^k, the next larger bf16 value the next power; a block of zeros the least."""
    c = Cache([0] * 8, [16] * 8, 2, 2, 64, 16, page=16, seed=1)
    c.k[:], c.v[:] = 0, 0
    tops = [448.0, 450.0, 1.75, 1.7578125, 224.0, -448.0, 0.0, 2.0 ** -126]
    for b, x in enumerate(tops):
        c.k[16 * b + b, 1, 3] = x
        c.v[16 * b + 15 - b, 0, 63] = x
    c.run().check()
    home = [int(c.rows_of(b)[0]) // 16 for b in range(8)]
    assert c.d_scale[0][home, 1].tolist() == [1.0, 2.0, 2.0 ** -8, 2.0 ** -7, 0.5, 1.0, 2.0 ** -60, 2.0 ** -60]


def test_older_codes_are_encoded_again_exactly():
    """All 256 codes under a scale 2^20 .. below what the new token asks for."""
    c = Cache([33], [1], 2, 2, 64, 64, page=64, seed=2)
    rows = c.rows_of(0)
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    for i in range(4):
        c.code[0][rows[8 * i], 0] = codes[64 * i:64 * i + 64]
    home = int(rows[0]) // 64
    for s in (2.0 ** -3, 2.0 ** -9, 2.0 ** -14, 2.0 ** -40):
        c.scale[0][home] = s
        c.run()
        code, scale, _, _ = c.expect()
        got = c.d_code[0].cpu()
        nan = (codes & 0x7F) == 0x7F
        for i in range(4):
            a, b = got[rows[8 * i], 0], code[0][rows[8 * i], 0]
            m = nan[64 * i:64 * i + 64]
            assert torch.equal(a[~m], b[~m]) and bool(((a[m] & 0x7F) == 0x7F).all())
        assert torch.equal(c.d_scale[0].cpu(), scale[0])


def test_values_that_are_not_finite():
    """They have no say in the scale; infinities saturate, NaN stays NaN."""
    c = Cache([10, 0], [8, 64], 2, 2, 64, 64, page=64, seed=4)
    c.k[2, 0, 5], c.k[3, 1, 6], c.v[1, 0, 7] = math.inf, -math.inf, math.nan
    c.v[8:72, 1] = math.nan  # a block and head of nothing else
    c.run()
    code, scale, _, _ = c.expect()
    for i in range(2):
        assert torch.equal(c.d_scale[i].cpu(), scale[i])
        a, b = c.d_code[i].cpu(), code[i]
        nan = (b & 0x7F) == 0x7F
        assert torch.equal(a[~nan], b[~nan]) and bool(((a[nan] & 0x7F) == 0x7F).all())


def test_tokens_one_by_one_or_at_once():
    """A block filled token by token holds what it would hold at once, but for values that fell below
    the smallest normal code when its scale grew: those are a step of the final scale off at most."""
    n, sb = 64, 64
    at_once = Cache([0], [n], 2, 2, 64, sb, page=64, seed=6, spare=0).run()
    c = Cache([0], [n], 2, 2, 64, sb, page=64, seed=6, spare=0)
    for i in range(n):
        one = Cache([i], [1], 2, 2, 64, sb, page=64, seed=6, spare=0)
        one.k, one.v, one.q = c.k[i:i + 1], c.v[i:i + 1], c.q[i:i + 1]
        one.code, one.scale = c.code, c.scale
        one.run().check()
        c.code, c.scale = [x.cpu() for x in one.d_code], [x.cpu() for x in one.d_scale]
    for i in range(2):
        assert torch.equal(c.scale[i], at_once.d_scale[i].cpu())
        x, y = BR.value_of(c.code[i]), BR.value_of(at_once.d_code[i].cpu())
        # each of up to 8 growths may round a subnormal value by half a step (2^-10) more
        assert bool(((x - y).abs() <= 8 * 2.0 ** -10).all())


def test_positions_of_minus_one_are_skipped():
    """What the plan refused: whole sequences, and single rows (their neighbours are stored)."""
    c = Cache([10, 20, 30], [3, 4, 5], 4, 2, 128, 64, page=64, seed=8)
    pos = list(c.pos)
    pos[3:7] = [-1] * 4
    c.run(pos=pos).check(skip=(1,))
    c = Cache([0], [20], 4, 2, 64, 16, page=16, seed=9)
    pos = list(c.pos)
    pos[16:] = [-1] * 4  # the second block has no token left: it stays as it was
    c.run(pos=pos)
    c.new, c.pos = [16], c.pos[:16]
    c.q_start = [0, 16]
    c.check()


def test_bad_tokens_are_reported_and_skipped():
    # positions that do not follow
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, page=64, seed=8)
    pos = list(c.pos)
    pos[5:7] = [25, 21]
    c.run(pos=pos, status=BAD)
    c.new, c.pos, c.q_start = [3, 2], pos[:5], [0, 3, 5]
    c.check()
    # a first position past the context
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, page=64, seed=8)
    pos = list(c.pos)
    pos[3:7] = [24, 25, 26, 27]
    c.run(pos=pos, status=BAD).check(skip=(1,))
    # a page outside the cache
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, page=64, seed=8)
    c.table[1, 0] = 1000
    c.run(status=BAD)
    c.table[1, 0] = 0  # (any place: the sequence is skipped)
    c.check(skip=(1,))
    # a contiguous sequence that does not start at a block
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, seed=8)
    c.base[1] += 1
    c.run(status=BAD).check(skip=(1,))
    # a malformed sequence
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, page=64, seed=8)
    c.run(ctx=[13, 2000000], status=0)  # (a longer context than the tokens: none of this call's business)
    c = Cache([10, 20], [3, 4], 4, 2, 128, 64, page=64, seed=8)
    c.run(ctx=[13, -1], status=BAD).check(skip=(1,))


def test_bad_older_scales_are_reported():
    for bad in (0.0, -1.0, math.inf, math.nan):
        c = Cache([10], [3], 2, 1, 64, 16, page=16, seed=8)
        home = int(c.rows_of(0)[0]) // 16
        c.scale[0][home, 0] = bad
        c.run(status=BAD)
        rows = c.rows_of(0)
        assert torch.equal(c.d_code[0].cpu()[rows[:10]], c.code[0][rows[:10]])
        s = BR.need_of(float(c.k.abs().max()))
        assert float(c.d_scale[0][home, 0]) == s
        assert torch.equal(c.d_code[0].cpu()[rows[10:]], BR.code_of(c.k.double() / s))


def test_without_queries_in_place_and_on_a_stream():
    c = Cache([10, 100], [70, 1], 8, 2, 128, 64, page=64, rot=64, half=True, seed=11)
    c.run(queries=False).check(queries=False)
    c.run(inplace=True).check()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.run(stream=st)
    c.check()


def test_the_same_bits_again():
    c = Cache([50, 1, 300], [200, 1, 9], 16, 4, 128, 32, page=64, rot=128, seed=12).run()
    first = [x.clone() for x in c.d_code + c.d_scale + [c.q_out]]
    for _ in range(5):
        c.run()
        assert all(torch.equal(a, b) for a, b in zip(first, c.d_code + c.d_scale + [c.q_out]))


# ---------------------------------------------------------------------------
# dense attention
DENSE = {
    # (contexts, new tokens, hq, hkv, d, page, scale block)
    "one token": ([1, 64, 65], [1, 1, 1], 8, 2, 128, 64, 64),
    "long": ([9001], [1], 16, 2, 128, 64, 16),
    "drafts": ([777, 20, 4, 130], [4, 4, 4, 4], 32, 4, 128, 64, 32),
    "contiguous": ([200, 33], [1, 2], 14, 2, 64, 0, 64),
    "pages of 256": ([1000, 257], [5, 1], 8, 8, 64, 256, 128),
    "prompts": ([333, 40], [333, 17], 8, 2, 128, 128, 128),
    "pages of 16": ([100, 40], [60, 1], 12, 4, 64, 16, 16),
}


def _block_scaled(c, sb, g):
    """The case's cache with a scale per block, and the same scales row by row."""
    n = -(-c.rows // sb)
    scales = [torch.exp2(torch.randint(-9, -5, (n, c.hkv), generator=g).float()) *
              (1 + 0.5 * torch.rand(n, c.hkv, generator=g)) for _ in range(2)]
    c.ks, c.vs = [s.repeat_interleave(sb, 0)[:c.rows].contiguous() for s in scales]
    return scales


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("name", DENSE)
def test_dense(name, call):
    """Against the 64-bit form, and the same bits as the same scales given row by row."""
    ctx, new, hq, hkv, d, page, sb = DENSE[name]
    c = Case(ctx, new, hq, hkv, d, e4m3=True, page=page, seed=len(name), dirty=False)
    scales = _block_scaled(c, sb, torch.Generator().manual_seed(1))
    c.dks, c.dvs = c.ks.to(DEV), c.vs.to(DEV)
    c.run(call).check()
    out, lse = c.out.clone(), c.lse.clone()
    c.shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_BLOCKSCALE, scale_block=sb)
    c.dks, c.dvs = scales[0].to(DEV), scales[1].to(DEV)
    c.run(call).check()
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse)

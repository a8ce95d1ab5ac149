"""Block bounds, block selection and attention over listed blocks on a GB300
through the C ABI, against the plain forms of block_reference.py (selection is
exact: whole numbers) and the error bounds of gqa_reference.py."""

from __future__ import annotations

import math

import pytest
import torch

import block_reference as BR
import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = dsa._binding.DSA_ERR_BAD_INPUT
KINDS = {"bf16": dsa.DSA_BF16, "row": dsa.DSA_FP8_E4M3_ROWSCALE, "block": dsa.DSA_FP8_E4M3_BLOCKSCALE}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Step:
    """Sequences over a cache (values of unused rows NaN), their bounds, and the calls."""

    def __init__(self, ctx, new, hq, hkv, d, block, *, kv="block", sb=0, page=0, nsel=4, first=0, local=1, seed=0,
                 extra_q=0, pos=None, q_gap=0, dirty=True, amp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.hq, self.hkv, self.d, self.block, self.page = ctx, new, hq, hkv, d, block, page
        self.kv, self.nsel, self.first, self.local = kv, nsel, first, local
        self.sb = sb or block
        B, unit = len(ctx), max(page, block, self.sb)
        used = [-(-n // (page or unit)) for n in ctx]
        order = torch.randperm(sum(used) + 2, generator=g)
        self.rows = (sum(used) + 2) * (page or unit)
        self.table = self.base = None
        if page:
            self.table = torch.full((B, max(used) + 1), -1, dtype=torch.int32)
            at = 0
            for b, u in enumerate(used):
                self.table[b, :u] = order[at:at + u].int()
                at += u
        else:
            self.base = [sum(used[:b]) * unit for b in range(B)]
        self.q_start = [0]
        for n in new:
            self.q_start.append(self.q_start[-1] + n)
        self.nq = self.q_start[-1]
        self.num_q = self.nq + extra_q
        self.pos = pos if pos is not None else [n - m + i for n, m in zip(ctx, new) for i in range(m)]
        self.seq = [b for b, m in enumerate(new) for _ in range(m)]
        self.q = (torch.randn(self.num_q, hq, d, generator=g) * amp).bfloat16()
        shape = (self.rows, hkv, d)
        if kv == "bf16":
            self.k, self.v = [(torch.randn(shape, generator=g) * amp).bfloat16() for _ in range(2)]
            self.ks = self.vs = self.kr = self.vr = None
        else:
            self.k, self.v = [(torch.randn(shape, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
                              .view(torch.uint8) for _ in range(2)]
            if kv == "row":
                self.ks, self.vs = [torch.rand(self.rows, hkv, generator=g) * 0.01 + 0.002 for _ in range(2)]
                self.kr, self.vr = self.ks, self.vs
            else:
                self.ks, self.vs = [torch.exp2(torch.randint(-9, -5, (self.rows // self.sb, hkv), generator=g).float())
                                    for _ in range(2)]
                self.kr, self.vr = [s.repeat_interleave(self.sb, 0) for s in (self.ks, self.vs)]
        live = torch.zeros(self.rows, dtype=torch.bool)
        for b, n in enumerate(ctx):
            live[R.rows_of(self.table, page, self.base, b, n)] = True
        if dirty:
            for x in (self.k, self.v):
                x[~live] = math.nan if kv == "bf16" else 0x7F
        n = self.rows // block
        self.bounds = torch.randint(-127, 128, (n, hkv, 2, d), generator=g).to(torch.int8)
        self.bounds = torch.stack([self.bounds.amin(2), self.bounds.amax(2)], 2).contiguous()
        self.steps = torch.exp2(torch.randint(-7, -3, (n, hkv), generator=g).float())
        self.sm_scale = 1.0 / math.sqrt(d)
        self.q_gap = q_gap
        self.seqs_args = dict(max_ctx=max(1, max(ctx)), max_q_per_seq=max(1, max(new)), num_rows=self.rows)
        self.device()

    def device(self):
        q = torch.zeros(self.num_q, self.hq + self.q_gap, self.d, dtype=torch.bfloat16, device=DEV)
        self.dq = q[:, :self.hq]
        self.dq.copy_(self.q)
        self.dk, self.dv = self.k.to(DEV), self.v.to(DEV)
        self.dks = None if self.ks is None else self.ks.to(DEV)
        self.dvs = None if self.vs is None else self.vs.to(DEV)
        self.dbounds, self.dsteps = self.bounds.to(DEV), self.steps.to(DEV)
        self.shape = dsa.GqaShape(self.hq, self.hkv, self.d, KINDS[self.kv], q_stride=self.dq.stride(0),
                                  scale_block=self.sb if self.kv == "block" else 0)
        self.seqs = dsa.Seqs(_i32(self.ctx), _i32(self.q_start), _i32(self.pos + [0] * (self.num_q - len(self.pos))),
                             page_table=None if self.table is None else self.table.to(DEV), page_size=self.page,
                             seq_base=None if self.base is None else torch.tensor(self.base, device=DEV),
                             **self.seqs_args)
        self.ws_bytes = dsa.block_gqa_workspace_size(self.shape, self.seqs, self.num_q, self.block, self.nsel)
        self.ws = torch.full((self.ws_bytes // 4 + 64,), math.nan, dtype=torch.float32, device=DEV).view(torch.uint8)
        self.status = _i32([0])
        self.blocks = torch.full((self.num_q, self.hkv, self.nsel), 77, dtype=torch.int32, device=DEV)
        self.len = torch.full((self.num_q, self.hkv), 77, dtype=torch.int32, device=DEV)
        self.out = torch.full((self.num_q, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.num_q, self.hq), 7.0, device=DEV)

    # ---- the calls
    def run_bounds(self, stream=None):
        dsa.block_gqa_bounds(self.shape, self.dk, self.dks, self.seqs, self.num_q, self.block, self.dbounds,
                             self.dsteps, d_status=self.status, stream=stream)
        return self

    def run_select(self, stream=None):
        dsa.block_gqa_select(self.shape, self.dq, self.dbounds, self.dsteps, self.seqs, self.num_q, self.block,
                             self.nsel, self.first, self.local, self.blocks, self.len, self.ws, self.ws_bytes,
                             d_status=self.status, stream=stream)
        return self

    def run_attend(self, stream=None, lse=True):
        dsa.block_gqa_attend(self.shape, self.dq, self.dk, self.dv, self.dks, self.dvs, self.seqs, self.num_q,
                             self.blocks, self.len, self.block, self.nsel, self.sm_scale, self.out,
                             self.lse if lse else None, self.ws, self.ws_bytes, d_status=self.status, stream=stream)
        return self

    def stat(self):
        torch.cuda.synchronize()
        return int(self.status)

    # ---- the plain forms
    def rows_of(self, b, n=None):
        return R.rows_of(self.table, self.page, self.base, b, self.ctx[b] if n is None else n)

    def values(self, which):
        x, s = (self.k, self.kr) if which == "k" else (self.v, self.vr)
        if s is None:
            return x.double()
        return (x.view(torch.float8_e4m3fn).float() * s[..., None]).double()  # an fp32 number, as the kernels see it

    def check_bounds(self, skip=(), status=0):
        assert self.stat() == status
        want, steps = self.bounds.clone(), self.steps.clone()
        k = self.values("k")
        for b, (n, m) in enumerate(zip(self.ctx, self.new)):
            if m == 0 or b in skip:
                continue
            p0 = self.pos[self.q_start[b]]
            if p0 < 0:
                continue
            rows = self.rows_of(b, p0 + m)
            for i in range(p0 // self.block, (p0 + m - 1) // self.block + 1):
                r = rows[i * self.block:(i + 1) * self.block]
                home = int(r[0]) // self.block
                want[home], steps[home] = BR.bounds_of(k[r])
        assert torch.equal(self.dsteps.cpu(), steps)
        assert torch.equal(self.dbounds.cpu(), want)

    def lists(self, t, g):
        """The plain form's blocks and keys of row t, key head g, from the bounds on the device."""
        pos, b = self.pos[t], self.seq[t]
        if pos < 0:
            return [], 0
        n = pos // self.block + 1
        rows = self.rows_of(b)
        home = torch.tensor([int(rows[i * self.block]) // self.block for i in range(n)])
        q = BR.whole(self.q[t, g * (self.hq // self.hkv):(g + 1) * (self.hq // self.hkv)].double())
        s = BR.scores(q, self.dbounds.cpu()[home, g], self.dsteps.cpu()[home, g])
        sel = BR.pick(s, n, self.nsel, self.first, self.local)
        return sel, (len(sel) - 1) * self.block + pos % self.block + 1

    def check_select(self, rows=None, status=0):
        assert self.stat() == status
        got, length = self.blocks.cpu(), self.len.cpu()
        for t in range(self.nq) if rows is None else rows:
            for g in range(self.hkv):
                sel, n = self.lists(t, g)
                assert got[t, g].tolist() == sel + [-1] * (self.nsel - len(sel)), (t, g)
                assert int(length[t, g]) == n
        assert bool((got[self.nq:] == 77).all()) and bool((length[self.nq:] == 77).all())

    def check_attend(self, rows=None, status=0, unwritten=()):
        assert self.stat() == status
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        k, v = R.values(self.k, self.kr), R.values(self.v, self.vr)
        blocks, length = self.blocks.cpu(), self.len.cpu()
        grp = self.hq // self.hkv
        for t in range(self.nq) if rows is None else rows:
            if t in unwritten:
                assert bool((out[t] == 7).all()) and bool((lse[t] == 7).all())
                continue
            at = self.rows_of(self.seq[t])
            for g in range(self.hkv):
                n = int(length[t, g])
                h = slice(g * grp, (g + 1) * grp)
                tok = [int(i) * self.block + x for i in blocks[t, g] for x in range(self.block)][:n]
                r = at[torch.tensor(tok, dtype=torch.long)]
                ref, rl, tol, ltol = R.attend(self.q[t:t + 1, h].double(), k[r, g:g + 1], v[r, g:g + 1], [n - 1],
                                              self.sm_scale)
                err = (out[t, h] - ref[0]).abs()
                assert bool((err <= tol[0]).all()), (t, g, float((err - tol[0]).max()))
                if n:
                    assert bool(((lse[t, h] - rl[0]).abs() <= ltol[0]).all()), (t, g)
                else:
                    assert bool((lse[t, h] == -math.inf).all())
        assert bool((out[self.nq:] == 7).all()) and bool((lse[self.nq:] == 7).all())


STEPS = {
    # (contexts, new, hq, hkv, d, block, kwargs)
    "one key": ([1], [1], 8, 1, 128, 64, dict()),
    "fewer blocks than the list": ([200, 65], [1, 1], 8, 2, 128, 64, dict(page=64, nsel=9)),
    "decode": ([1000, 333, 64, 63], [1, 1, 1, 1], 16, 2, 128, 64, dict(page=64, nsel=5, first=1, local=2)),
    "drafts": ([1000, 333, 66, 5], [4, 4, 4, 4], 16, 2, 128, 16, dict(page=64, nsel=8, sb=64)),
    "bf16": ([700, 1300], [2, 1], 12, 4, 128, 32, dict(kv="bf16", page=32, nsel=6, local=2)),
    "bf16 d64 contiguous": ([700, 1300], [2, 1], 5, 5, 64, 64, dict(kv="bf16", nsel=3, first=2)),
    "row scales": ([700, 1300], [2, 1], 14, 2, 128, 128, dict(kv="row", page=256, nsel=4)),
    "row scales d64": ([700], [1], 6, 3, 64, 16, dict(kv="row", page=16, nsel=11, first=3, local=4)),
    "group of 16": ([900], [3], 32, 2, 128, 64, dict(page=128, nsel=4, sb=16)),
    "group of 33": ([500], [2], 33, 1, 64, 32, dict(page=64, nsel=4, sb=32)),
    "group of 64": ([300], [2], 64, 1, 128, 16, dict(page=64, nsel=4, sb=64)),
    "ungrouped": ([400, 90], [5, 1], 7, 7, 64, 16, dict(page=16, nsel=5)),
    "pairs": ([400, 90], [5, 1], 4, 2, 128, 64, dict(kv="bf16", page=64, nsel=2)),
    "groups of 3": ([400], [7], 9, 3, 128, 32, dict(page=64, nsel=4, sb=16)),
    "prompt": ([300], [300], 8, 2, 128, 16, dict(page=64, nsel=6, first=1, local=2, sb=64)),
    "ragged prompts": ([150, 20, 400, 7], [150, 3, 61, 0], 8, 2, 64, 32, dict(page=64, nsel=4, sb=64)),
    "many blocks": ([60000], [1], 8, 1, 64, 16, dict(kv="bf16", page=64, nsel=64, first=1, local=2)),
    "prompt of group 20": ([260], [200], 20, 1, 128, 32, dict(page=64, nsel=4, sb=64)),
    "prompt of group 33": ([260], [130], 33, 1, 64, 16, dict(kv="bf16", page=64, nsel=4)),
    "ungrouped prompt": ([1500], [700], 3, 3, 64, 16, dict(kv="bf16", page=64, nsel=7, first=1)),
    "prompt of many tiles": ([9000], [37], 8, 1, 128, 16, dict(kv="bf16", page=64, nsel=40, first=1, local=2)),
    "many sequences": ([900 - 5 * i for i in range(160)], [1 + i % 3 for i in range(160)], 8, 2, 128, 16,
                       dict(kv="bf16", page=64, nsel=9, first=1, local=2)),
    "many sequences of drafts": ([300 + 3 * i for i in range(80)], [4] * 80, 20, 4, 64, 16,
                                 dict(kv="bf16", page=16, nsel=7)),
    "many rows": ([1500], [1400], 8, 4, 64, 16, dict(kv="bf16", page=64, nsel=9, first=1, local=2)),
    "many rows, more blocks": ([8000], [1300], 4, 4, 64, 16, dict(kv="bf16", page=64, nsel=33)),
    "many rows, most blocks": ([16000], [1250], 4, 4, 64, 16, dict(kv="bf16", page=64, nsel=200, first=2, local=3)),
    "a list of one": ([400, 16], [2, 1], 8, 2, 64, 16, dict(page=16, nsel=1)),
    "nothing but sure ones": ([400], [2], 8, 2, 64, 16, dict(page=16, nsel=5, first=2, local=3)),
    "a list of 200": ([9000], [2], 8, 1, 64, 16, dict(page=16, nsel=200)),
}


def _step(name, **kw):
    ctx, new, hq, hkv, d, block, args = STEPS[name]
    return Step(ctx, new, hq, hkv, d, block, seed=len(name), **{"extra_q": 2, "q_gap": 1, **args, **kw})


def _few(s, n=40):
    return None if s.nq <= n else sorted({0, 1, s.nq - 1} | {i * s.nq // n for i in range(n)})


@pytest.mark.parametrize("name", STEPS)
def test_bounds(name):
    _step(name).run_bounds().check_bounds()


@pytest.mark.parametrize("name", STEPS)
def test_select(name):
    s = _step(name).run_select()
    s.check_select(_few(s))


@pytest.mark.parametrize("name", STEPS)
def test_bounds_select_attend(name):
    """The three as a layer runs them."""
    s = _step(name).run_bounds().run_select().run_attend()
    s.check_select(_few(s))
    s.check_attend(_few(s))


# ---------------------------------------------------------------------------
def test_bounds_hold():
    """A block's score is no less than any of its keys' scores with the queries in whole steps."""
    s = Step([512], [512], 8, 2, 64, 16, kv="bf16", page=64, seed=3).run_bounds()
    assert s.stat() == 0
    k = s.values("k")[s.rows_of(0)]
    rows = s.rows_of(0)
    for t in range(0, 512, 37):
        for g in range(2):
            home = torch.tensor([int(rows[i * 16]) // 16 for i in range(32)])
            qf = s.q[t, 4 * g:4 * g + 4].double()
            q = BR.whole(qf)
            score = BR.scores(q, s.dbounds.cpu()[home, g], s.dsteps.cpu()[home, g])
            best = (q @ k[:, g].T).amax(0).view(32, 16).amax(1)
            assert bool((score >= best).all())


def test_bounds_at_borders_and_of_values_that_are_not_finite():
    s = Step([16 * 9], [16 * 9], 2, 1, 64, 16, kv="bf16", page=16, seed=1)
    rows = s.rows_of(0)
    s.k[rows] = 0
    tops = [127.0, 127.5, 254.0, -127.0, 0.0, 2.0 ** -130, 3e38, 1.0]
    for i, x in enumerate(tops):
        s.k[rows[16 * i + i], 0, 5] = x
        s.k[rows[16 * i + i + 1], 0, 5] = -x / 4
    last = rows[16 * 8:]
    s.k[last[0], 0, 0], s.k[last[1], 0, 1], s.k[last[2], 0, 2], s.k[last[3], 0, 3] = math.inf, -math.inf, math.nan, 2.0
    s.k[rows[16 * 7 + 3], 0, 9] = -2.0 ** -120  # far below a step: still below 0
    s.device()
    s.run_bounds().check_bounds()


@pytest.mark.parametrize("kv", ["row", "block"])
@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_codes_and_scales_of_any_kind(kv, d):
    """NaN codes, and scales that are negative, zero or not finite."""
    s = Step([16 * 8], [16 * 8], 3, 3, d, 16, kv=kv, page=16, seed=1)
    rows = s.rows_of(0)
    s.k[rows[5], 0, 3], s.k[rows[16 + 7], 1, d - 1] = 0x7F, 0xFF
    at = rows if kv == "row" else rows // 16
    for i, x in enumerate([-0.25, 0.0, math.inf, -math.inf, math.nan, 2.0 ** -126]):
        s.ks[at[16 * (i + 2) + (3 if kv == "row" else 0)], 0] = x
    s.kr = s.ks if kv == "row" else s.ks.repeat_interleave(16, 0)
    s.device()
    s.run_bounds().check_bounds()


@pytest.mark.parametrize("tokens", [1, 700])
def test_nothing_but_padding(tokens):
    """Rows behind the last sequence alone: nothing is written."""
    s = Step([400, 50], [tokens, 1], 8, 2, 64, 16, page=16, extra_q=3)
    s.blocks.fill_(0)
    s.len.fill_(16)
    s.seqs.q_start = _i32([0, 0, 0])
    s.run_bounds().run_select().run_attend()
    assert s.stat() == 0
    assert bool((s.out == 7).all()) and bool((s.lse == 7).all()) and bool((s.blocks == 0).all())
    assert torch.equal(s.dbounds.cpu(), s.bounds)


def test_queries_that_are_not_finite_or_zero():
    s = Step([500] * 4, [1] * 4, 8, 2, 64, 16, kv="bf16", page=16, nsel=5, seed=2)
    s.q[0] = 0
    s.q[1, 3, 7], s.q[1, 6, 7] = math.inf, -math.inf
    s.q[2, 1, 1] = math.nan
    s.q[3] = math.nan
    s.device()
    s.run_select().check_select()


def test_equal_scores_go_to_the_smaller_block():
    """Few distinct scores over many blocks, the cut in the middle of a tie."""
    for seed in range(4):
        s = Step([64 * 700], [1], 8, 2, 64, 64, kv="bf16", page=64, nsel=100, first=1, local=2, seed=seed)
        s.bounds[:] = 0
        g = torch.Generator().manual_seed(seed)
        s.bounds[:, :, 1, :] = torch.randint(0, 1 + seed, s.steps.shape, generator=g).to(torch.int8)[..., None]
        s.steps[:] = 1.0
        s.device()
        s.run_select().check_select()


@pytest.mark.parametrize("nsel", [6, 100, 300])
@pytest.mark.parametrize("new, levels", [(1300, 1), (1300, 2), (1300, 40), (40, 2)])
def test_equal_scores_in_many_rows(new, levels, nsel):
    """The cut inside ties for rows that a warp chooses, with few keys left and with many."""
    s = Step([12000], [new], 4, 4, 64, 16, kv="bf16", page=64, nsel=nsel, first=1, local=2, seed=levels)
    s.bounds[:] = 0
    g = torch.Generator().manual_seed(levels)
    s.bounds[:, :, 1, :] = torch.randint(0, levels, s.steps.shape, generator=g).to(torch.int8)[..., None]
    s.steps[:] = 1.0
    s.device()
    s.run_select().check_select(_few(s, 10))


def test_steps_that_were_never_written():
    """NaN scores come last, whatever chooses (few rows, many rows, long rows): the lists are whole."""
    for ctx, new, nsel in ((16 * 300, 1, 30), (16 * 300, 1300, 30), (16 * 300, 1300, 290), (16 * 5000, 1, 30)):
        s = Step([ctx], [new], 4, 4, 64, 16, kv="bf16", page=16, nsel=nsel, first=1, seed=5)
        s.steps[::3] = math.nan
        s.device()
        s.run_select()
        assert s.stat() == 0
        got = s.blocks[s.nq - 1].cpu()
        rows = s.rows_of(0)
        bad = {i for i in range(ctx // 16) if int(rows[16 * i]) // 16 % 3 == 0}
        for g in range(4):
            sel = got[g].tolist()
            assert sel == sorted(set(sel)) and len(sel) == nsel and sel[0] == 0 and sel[-1] == ctx // 16 - 1
            want = max(0, nsel - (ctx // 16 - len(bad)) - 2)
            assert len(bad & set(sel)) <= want + 2


def test_steps_far_apart():
    s = Step([16 * 300], [1], 8, 2, 64, 16, kv="bf16", page=16, nsel=30, seed=5)
    s.steps[:] = torch.exp2(torch.randint(-100, 80, s.steps.shape, generator=torch.Generator().manual_seed(1)).float())
    s.device()
    s.run_select().check_select()


@pytest.mark.parametrize("n", [1025, 4097, 51200])
def test_long_rows(n):
    """Up to the most blocks that are served."""
    s = Step([16 * n], [1], 2, 1, 64, 16, kv="bf16", page=256, nsel=33, first=1, seed=n)
    s.run_select().check_select()


def test_positions_of_minus_one_and_bad_ones():
    pos = [899, -1, 400, 63, -1]
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32, nsel=4, pos=[898, -1, 400, 401, -1], extra_q=1)
    s.run_select().run_attend()
    s.check_select()
    s.check_attend()
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32, nsel=4, pos=[898, 900, -2, 401, 63], extra_q=1)
    s.run_select()
    s.check_select(rows=[0, 3, 4], status=BAD)
    for t in (1, 2):
        assert bool((s.blocks[t] == 77).all()) and bool((s.len[t] == 77).all())
    del pos


def test_bounds_skip_and_report():
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32, pos=[898, 899, -1, -1, 63])
    s.run_bounds().check_bounds()
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32, pos=[898, 899, 499, 500, 63])
    s.run_bounds().check_bounds(skip=(1,), status=BAD)
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32)
    s.seqs.page_table[1, 15] = 9999
    s.run_bounds().check_bounds(skip=(1,), status=BAD)
    s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32)
    s.seqs.seq_base[1] += 4
    s.run_bounds().check_bounds(skip=(1,), status=BAD)


def test_malformed_sequences():
    for kw in (dict(ctx=[900, -1, 64]), dict(q_start=[0, 3, 2, 5]), dict(q_start=[0, 2, 9, 5])):
        s = Step([900, 500, 64], [2, 2, 1], 8, 2, 64, 32, page=32)
        if "ctx" in kw:
            s.seqs.ctx_len = _i32(kw["ctx"])
        else:
            s.seqs.q_start = _i32(kw["q_start"])
        s.blocks[:], s.len[:] = -1, 0
        s.blocks[:, :, 0], s.len[:] = 0, 5
        s.run_attend()
        s.run_bounds()
        s.run_select()
        assert s.stat() == BAD


def _random_lists(s, seed=0, empty=True):
    """Any lists: in any order, any number of keys."""
    g = torch.Generator().manual_seed(seed)
    blocks = torch.full((s.num_q, s.hkv, s.nsel), -1, dtype=torch.int32)
    length = torch.zeros(s.num_q, s.hkv, dtype=torch.int32)
    for t in range(s.nq):
        n = s.ctx[s.seq[t]] // s.block  # whole blocks
        for h in range(s.hkv):
            m = int(torch.randint(0 if empty else 1, min(s.nsel, n) + 1, (1,), generator=g))
            blocks[t, h, :m] = torch.randperm(n, generator=g)[:m].int()
            length[t, h] = m * s.block - (int(torch.randint(0, s.block, (1,), generator=g)) if m else 0)
    s.blocks, s.len = blocks.to(DEV), length.to(DEV)


@pytest.mark.parametrize("name", ["decode", "drafts", "bf16", "row scales", "row scales d64", "group of 16",
                                  "group of 64", "ungrouped", "groups of 3"])
def test_any_lists(name):
    """Lists that differ between the heads in order, length and number, empty ones among them."""
    s = _step(name)
    _random_lists(s, seed=len(name))
    s.run_attend().check_attend()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("tokens, nsel", [(1, 32), (3, 40), (40, 32), (700, 8), (2000, 3)])
def test_splits_and_joins(kv, tokens, nsel):
    """Clusters, cut lists and the joining kernel, whole lists in turn, by the number of tokens."""
    s = Step([4000] * tokens if tokens < 100 else [4000], [1] * tokens if tokens < 100 else [tokens], 8, 2, 128, 64,
             kv=kv, page=64, nsel=nsel, seed=tokens, extra_q=1)
    _random_lists(s, seed=tokens, empty=False)
    s.run_attend().check_attend(_few(s, 12))


def test_the_same_block_twice():
    """It counts twice: the same weights, so lse grows by ln 2 and out stays, up to their roundings."""
    s = Step([640], [1], 8, 2, 64, 64, page=64, nsel=2)
    s.blocks[:], s.len[:] = 3, 128
    s.run_attend().check_attend()


def test_bad_lists():
    s = Step([640, 200], [1, 1], 8, 2, 64, 64, kv="bf16", page=64, nsel=4, dirty=False)
    s.blocks[:], s.len[:] = torch.tensor([0, 1, 2, -1], device=DEV, dtype=torch.int32), 192
    s.len[0, 0] = 257  # more than the list holds
    s.run_attend()
    assert s.stat() == BAD
    assert bool((s.out[0, :4] == 7).all())
    s.nq = 2
    for x in (-1, 4, 1 << 30, -(1 << 31)):  # sequence 1 has four blocks: 0 .. 3
        s = Step([640, 200], [1, 1], 8, 2, 64, 64, kv="bf16", page=64, nsel=4, dirty=False)
        s.blocks[:], s.len[:] = torch.tensor([0, x, 2, -1], device=DEV, dtype=torch.int32), 192
        s.blocks[0, :, 1] = 1
        s.run_attend()
        # that block's keys and values count as zeros
        s.k = torch.cat([s.k, torch.zeros(64, 2, 64, dtype=torch.bfloat16)])
        s.v = torch.cat([s.v, torch.zeros(64, 2, 64, dtype=torch.bfloat16)])
        spare = s.rows
        keep = s.rows_of

        def rows_of(b, n=None, keep=keep, spare=spare):
            r = keep(b, 256 if b == 1 else n).clone()
            if b == 1:
                r[64:128] = torch.arange(spare, spare + 64)
            return r
        s.rows_of = rows_of
        s.table = torch.where(s.table < 0, torch.zeros_like(s.table), s.table)
        s.blocks[1, :, 1] = 1
        s.check_attend(status=BAD)
    s = Step([640], [1], 8, 2, 64, 64, page=64, nsel=2)
    s.blocks[:], s.len[:] = 0, -1
    s.run_attend().check_attend(status=BAD, unwritten=(0,))


def test_all_blocks_give_the_dense_result():
    s = Step([500, 320], [3, 1], 16, 2, 128, 64, kv="bf16", page=64, nsel=8).run_select().run_attend()
    assert s.stat() == 0
    out, lse = s.out.double(), s.lse.double()
    dense = torch.empty_like(s.out), torch.empty_like(s.lse)
    n = dsa.dense_gqa_workspace_size(s.shape, s.seqs, s.num_q)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dsa.dense_gqa_decode(s.shape, s.dq, s.dk, s.dv, None, None, s.seqs, s.num_q, s.sm_scale, dense[0], dense[1], ws, n)
    torch.cuda.synchronize()
    # both within the roundings of weights and results (2^-8 each of the largest value)
    assert float((out - dense[0].double()).abs().max()) <= 2 * 2.0 ** -7 * float(s.dv.double().abs().nan_to_num().max())
    assert float((lse - dense[1].double()).abs().max()) <= 1e-4


def test_no_lse_negative_scale_and_streams():
    s = _step("decode").run_bounds().run_select()
    s.sm_scale = -s.sm_scale
    s.run_attend(lse=False)
    s.lse[:] = 7
    first = s.out.clone()
    s.run_attend().check_attend()
    assert torch.equal(first, s.out)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    s.blocks.fill_(77)
    torch.cuda.synchronize()
    s.run_bounds(st).run_select(st).run_attend(st)
    s.check_select()
    assert torch.equal(first, s.out)


def test_the_same_bits_again():
    s = _step("ragged prompts").run_bounds().run_select().run_attend()
    assert s.stat() == 0
    first = [x.clone() for x in (s.dbounds, s.dsteps, s.blocks, s.len, s.out, s.lse)]
    for _ in range(10):
        s.run_bounds().run_select().run_attend()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (s.dbounds, s.dsteps, s.blocks, s.len, s.out, s.lse)))

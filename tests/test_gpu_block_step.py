"""A serving step of a layer over an 8-bit cache as a server runs it: the plan,
the writes, dense attention or the bounds, the selection and attention over the
selected blocks; step after step, captured into a graph, and two at once."""

from __future__ import annotations

import math

import pytest
import torch

import block_reference as BR
import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


class Server:
    """B requests over a paged cache; a step appends tokens and attends."""

    def __init__(self, B, hq=8, hkv=2, d=64, page=32, sb=16, block=16, nsel=4, max_ctx=512, max_new=64, rows=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.d, self.page, self.sb = B, hq, hkv, d, page, sb
        self.block, self.nsel, self.rows, self.max_new, self.max_ctx = block, nsel, rows, max_new, max_ctx
        self.num_pages = B * (max_ctx // page)
        self.free = torch.randperm(self.num_pages, generator=g).int().to(DEV)
        self.range = [torch.tensor([0, self.num_pages], dtype=torch.int32, device=DEV),
                      torch.zeros(2, dtype=torch.int32, device=DEV)]
        i32 = dict(dtype=torch.int32, device=DEV)
        self.table = torch.full((B, max_ctx // page), -1, **i32)
        self.cached, self.new = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.ctx, self.q_start, self.q_pos = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(rows, **i32)
        self.slot = torch.zeros(rows, dtype=torch.int64, device=DEV)
        n = self.num_pages * page
        self.kc, self.vc = [torch.full((n, hkv, d), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.ks, self.vs = [torch.full((n // sb, hkv), math.nan, device=DEV) for _ in range(2)]
        self.bounds = torch.zeros(n // block, hkv, 2, d, dtype=torch.int8, device=DEV)
        self.steps = torch.full((n // block, hkv), math.nan, device=DEV)
        self.x = torch.zeros(rows, hq + 2 * hkv, d, dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV)
        self.inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
        self.shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_BLOCKSCALE, scale_block=sb)
        self.seqs = dsa.Seqs(self.ctx, self.q_start, self.q_pos, max_ctx=max_ctx, max_q_per_seq=max_new,
                             num_rows=n, page_table=self.table, page_size=page)
        self.blocks = torch.zeros(rows, hkv, nsel, **i32)
        self.len = torch.zeros(rows, hkv, **i32)
        self.out = [torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        self.lse = [torch.zeros(rows, hq, device=DEV) for _ in range(3)]
        self.wb = dsa.block_gqa_workspace_size(self.shape, self.seqs, rows, block, nsel)
        self.wd = dsa.dense_gqa_workspace_size(self.shape, self.seqs, rows)
        self.ws = torch.empty(max(self.wb, self.wd), dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(1, **i32)
        self.scale = 1 / math.sqrt(d)
        # what a host keeps of it
        self.k = [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(B)]
        self.v = [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(B)]

    def enqueue(self):
        """Every call of the step, on the current stream."""
        st = self.status
        dsa.dsa_step_plan(self.cached, self.new, self.B, self.free, self.range[0], self.page, self.num_pages, self.table,
                          self.rows, self.ctx, self.q_start, self.q_pos, self.slot, self.range[1], d_status=st)
        q, k, v = self.x[:, :self.hq], self.x[:, self.hq:self.hq + self.hkv], self.x[:, self.hq + self.hkv:]
        dsa.dsa_kv_block_insert(self.shape, k, v, q, self.seqs, self.rows, self.inv, self.d, dsa.DSA_ROPE_HALVES, self.kc,
                                self.vc, self.ks, self.vs, self.q, k_stride=k.stride(0), v_stride=v.stride(0),
                                q_stride=q.stride(0), d_status=st)
        dsa.block_gqa_bounds(self.shape, self.kc, self.ks, self.seqs, self.rows, self.block, self.bounds, self.steps,
                             d_status=st)
        dsa.block_gqa_select(self.shape, self.q, self.bounds, self.steps, self.seqs, self.rows, self.block, self.nsel, 1,
                             1, self.blocks, self.len, self.ws, self.ws.numel(), d_status=st)
        dsa.block_gqa_attend(self.shape, self.q, self.kc, self.vc, self.ks, self.vs, self.seqs, self.rows, self.blocks,
                             self.len, self.block, self.nsel, self.scale, self.out[0], self.lse[0], self.ws,
                             self.ws.numel(), d_status=st)
        for i, call in ((1, dsa.dense_gqa_decode), (2, dsa.dense_gqa_prefill)):
            call(self.shape, self.q, self.kc, self.vc, self.ks, self.vs, self.seqs, self.rows, self.scale, self.out[i],
                 self.lse[i], self.ws, self.ws.numel(), d_status=st)
        # the next step's lengths and free pages
        self.cached.copy_(self.ctx)
        self.range[0].copy_(self.range[1])

    def load(self, new, seed):
        """New tokens' projections; the host's own copies of what the cache will hold."""
        g = torch.Generator().manual_seed(seed)
        n = sum(new)
        x = torch.randn(self.rows, self.hq + 2 * self.hkv, self.d, generator=g).bfloat16()
        self.x.copy_(x)
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        at, self.rows_of = 0, []
        for b, m in enumerate(new):
            past = self.k[b].shape[0]
            pos = torch.arange(past, past + m)
            part = x[at:at + m].double()
            k = R.rotate(part[:, self.hq:self.hq + self.hkv], pos, self.inv.cpu(), self.d, True)
            self.k[b] = torch.cat([self.k[b], k])
            self.v[b] = torch.cat([self.v[b], part[:, self.hq + self.hkv:]])
            q = R.rotate(part[:, :self.hq], pos, self.inv.cpu(), self.d, True)
            self.rows_of.append((at, m, past, q))
            at += m
        self.used = n

    def check(self):
        """Against attention over the exact keys and values: beside the kernels' own roundings, codes are
        within half a step (2^-4) of them, or 2^-10 of a block's scale (at most 2^-7 of its largest value
        here, 2 / 448 of it) where subnormal: values enter out with that error, keys move a score by it."""
        torch.cuda.synchronize()
        assert int(self.status) == 0
        assert int(self.range[0][0]) == sum(-(-k.shape[0] // self.page) for k in self.k)
        out, lse = [o.double().cpu() for o in self.out], [x.double().cpu() for x in self.lse]
        blocks, length = self.blocks.cpu(), self.len.cpu()
        grp = self.hq // self.hkv
        for b, (at, m, past, q) in enumerate(self.rows_of):
            for i in sorted({0, m // 2, m - 1}) if m else []:
                n = past + i + 1
                for h in range(self.hq):
                    g = h // grp
                    want = n if n <= self.nsel * self.block else None
                    for kind in range(3):
                        tok = torch.arange(n)
                        if kind == 0:
                            sel = blocks[at + i, g].tolist()
                            if want:
                                assert [x for x in sel if x >= 0] == list(range(-(-n // self.block)))
                            assert sel[0] == 0 and max(sel) == (n - 1) // self.block
                            tok = torch.cat([torch.arange(x * self.block, (x + 1) * self.block) for x in sel if x >= 0])
                            tok = tok[:int(length[at + i, g])]
                            assert int(tok[-1]) == n - 1
                        k, v = self.k[b][tok, g], self.v[b][tok, g]
                        s = self.scale * (k @ q[i, h])
                        p = torch.softmax(s, 0)
                        size = 2.0 ** -4 * k.abs() + 2.0 ** -16 * k.abs().max()
                        ds = float((self.scale * (size @ q[i, h].abs())).max()) + 2.0 ** -7 * float(s.abs().max())
                        top = float(v.abs().max())
                        tol = (math.exp(2 * ds) - 1 + 2.0 ** -4 + 2.0 ** -6) * (p @ v.abs()) + 2.0 ** -9 * top
                        assert bool(((out[kind][at + i, h] - p @ v).abs() <= tol).all()), (b, i, h, kind)
                        assert abs(float(lse[kind][at + i, h] - torch.logsumexp(s, 0))) <= ds + 1e-3


STEPS = [[20, 3, 0, 7], [1, 1, 40, 1], [1, 1, 1, 1], [4, 4, 4, 4], [1, 0, 1, 33], [1, 1, 1, 1], [30, 1, 1, 1]]


def test_steps_one_after_another():
    s = Server(4)
    for i, new in enumerate(STEPS):
        s.load(new, i)
        s.enqueue()
        s.check()


def test_a_captured_step_replayed():
    """The same graph for steps of different lengths, and the same bits as without it."""
    s, e = Server(4), Server(4)
    st = torch.cuda.Stream()
    graph = None
    for i, new in enumerate(STEPS):
        e.load(new, i)
        e.enqueue()
        s.load(new, i)
        torch.cuda.synchronize()
        if graph is None:
            state = [x.clone() for x in (s.cached, s.range[0], s.range[1], s.table, s.kc, s.vc, s.ks, s.vs, s.bounds,
                                         s.steps, s.ctx)]
            with torch.cuda.stream(st):
                s.enqueue()  # the kernels' first calls set their attributes
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    s.enqueue()
            for x, y in zip((s.cached, s.range[0], s.range[1], s.table, s.kc, s.vc, s.ks, s.vs, s.bounds, s.steps,
                             s.ctx), state):
                x.copy_(y)
        graph.replay()
        s.check()
        for x, y in zip(s.out + s.lse + [s.q], e.out + e.lse + [e.q]):
            assert torch.equal(x[:s.used], y[:s.used])
        for x, y in zip((s.kc, s.vc, s.bounds, s.blocks[:s.used], s.len[:s.used], s.table, s.q_pos, s.slot),
                        (e.kc, e.vc, e.bounds, e.blocks[:s.used], e.len[:s.used], e.table, e.q_pos, e.slot)):
            assert torch.equal(x, y)


def test_two_steps_at_once():
    """Two servers on two streams, each with its own workspace, hundreds of calls in flight."""
    a, b = Server(3, seed=1), Server(4, hq=16, seed=2)
    ref = {}
    for name, s, new in (("a", a, [30, 1, 20]), ("b", b, [1, 40, 3, 9])):
        s.load(new, 5)
        s.enqueue()
        torch.cuda.synchronize()
        # from here on the same tokens again: lengths as they were before
        s.cached.zero_()
        s.range[0].copy_(torch.tensor([0, s.num_pages], dtype=torch.int32))
        s.enqueue()
        torch.cuda.synchronize()
        ref[name] = [x.clone() for x in s.out + s.lse]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(40):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.cached.zero_()
                s.range[0].copy_(torch.tensor([0, s.num_pages], dtype=torch.int32))
                s.enqueue()
    torch.cuda.synchronize()
    assert int(a.status) == 0 and int(b.status) == 0
    for name, s in (("a", a), ("b", b)):
        assert all(torch.equal(x[:s.used], y[:s.used]) for x, y in zip(ref[name], s.out + s.lse))


def test_refused_requests_leave_the_others_alone():
    """Pages run out in the middle: the refused requests' rows are zeros, nothing of theirs is stored."""
    s = Server(4, rows=95)
    s.range[0].copy_(torch.tensor([0, 3], dtype=torch.int32))
    before = s.kc.clone()
    s.load([20, 60, 10, 5], 3)  # one, two, one and one page
    s.enqueue()
    torch.cuda.synchronize()
    assert int(s.status) == dsa._binding.DSA_ERR_BAD_INPUT
    assert s.ctx.tolist() == [20, 60, 0, 0] and s.range[1].tolist() == [3, 3]
    assert s.q_pos.tolist() == list(range(20)) + list(range(60)) + [-1] * 15
    for out, lse in zip(s.out, s.lse):
        assert bool((out[80:95] == 0).all()) and bool((lse[80:95] == -math.inf).all())
        assert bool((out[:80] != 0).any(-1).all())
    rest = torch.ones(s.kc.shape[0], dtype=torch.bool, device=DEV)
    rest[s.slot[:80]] = False
    assert torch.equal(s.kc[rest], before[rest])


def test_lists_of_the_plan_serve_the_other_writes():
    """dsa_kv_insert with the plan's positions and slots, padding rows among them."""
    s = Server(3)
    s.load([5, 17, 1], 0)
    dsa.dsa_step_plan(s.cached, s.new, s.B, s.free, s.range[0], s.page, s.num_pages, s.table, s.rows, s.ctx, s.q_start,
                      s.q_pos, s.slot, s.range[1], d_status=s.status)
    shape = dsa.GqaShape(s.hq, s.hkv, s.d)
    n = s.kc.shape[0]
    k, v = [torch.zeros(n, s.hkv, s.d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    x = s.x
    kk, vv = x[:, s.hq:s.hq + s.hkv].contiguous(), x[:, s.hq + s.hkv:].contiguous()
    dsa.dsa_kv_insert(shape, kk, vv, None, s.q_pos, s.slot, s.rows, None, 0, dsa.DSA_ROPE_PAIRS, k, v, None, None, n,
                      None, d_status=s.status)
    torch.cuda.synchronize()
    assert int(s.status) == 0
    assert torch.equal(k[s.slot[:23]], kk[:23]) and torch.equal(v[s.slot[:23]], vv[:23])
    assert int((k != 0).any(-1).any(-1).sum()) == 23


def test_value_of_code_is_the_torch_type():
    assert float(BR.value_of(BR.code_of(torch.tensor([448.0], dtype=torch.float64)))[0]) == 448.0

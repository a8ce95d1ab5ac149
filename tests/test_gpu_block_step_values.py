"""Serving steps over an 8-bit cache, every result against the formula of the
call that made it, from what the cache holds at that moment: codes and scales of
the writes, bounds, lists, and the three attentions within their kernels' own
roundings (a wrong block, scale or key does not fit in those)."""

from __future__ import annotations

import pytest
import torch

import block_reference as BR
import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R
from test_gpu_block_step import STEPS, Server

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


class Checked(Server):
    def before(self):
        torch.cuda.synchronize()
        return [x.cpu().clone() for x in (self.kc, self.ks, self.vc, self.vs)]

    def place(self, b, n):
        return R.rows_of(self.table.cpu(), self.page, None, b, n)

    def check_writes(self, old):
        """The plain write applied to what the cache held before: values' codes and all scales equal, keys
        within half a step of e4m3 and the rotation's fp32 roundings (as of the write's own tests)."""
        kc, ks, vc, vs = old
        got = self.before()
        fresh = torch.zeros(kc.shape[0], dtype=torch.bool)
        for b, (at, m, past, q) in enumerate(self.rows_of):
            if m == 0:
                continue
            rows = self.place(b, past + m)
            k, v = self.k[b][past:], self.v[b][past:]
            BR.insert(k, kc, ks, rows, past, self.sb)
            BR.insert(v, vc, vs, rows, past, self.sb)
            new = rows[past:]
            fresh[new] = True
            sc = ks[new // self.sb].double()[..., None]
            x = self.x[at:at + m, self.hq:self.hq + self.hkv].double().cpu()
            tol = 2.0 ** -4 * k.abs() + 2.0 ** -10 * sc + 2.0 ** -19 * x.abs().amax(-1, keepdim=True)
            assert bool(((BR.value_of(got[0][new]) * sc - k).abs() <= tol).all())
            x = self.x[at:at + m, :self.hq].double().cpu()
            err = (self.q[at:at + m].double().cpu() - q).abs()
            assert bool((err <= 2.0 ** -8 * q.abs() + 2.0 ** -19 * x.abs().amax(-1, keepdim=True)).all())
        used = torch.cat([self.place(b, past + m) for b, (at, m, past, q) in enumerate(self.rows_of)])
        home = used // self.sb
        assert torch.equal(got[1][home], ks[home]) and torch.equal(got[3][home], vs[home])
        assert torch.equal(got[2][used], vc[used])
        assert torch.equal(got[0][~fresh], kc[~fresh])

    def check_rest(self):
        """Bounds, lists and outputs from the cache, the bounds and the queries on the device."""
        kc, ks, vc, vs = self.before()
        k = BR.value_of(kc) * ks.double().repeat_interleave(self.sb, 0)[..., None]
        v = BR.value_of(vc) * vs.double().repeat_interleave(self.sb, 0)[..., None]
        bounds, steps, blocks, length = [x.cpu() for x in (self.bounds, self.steps, self.blocks, self.len)]
        out, lse = [o.double().cpu() for o in self.out], [x.double().cpu() for x in self.lse]
        query = self.q.double().cpu()
        grp = self.hq // self.hkv
        for b, (at, m, past, _) in enumerate(self.rows_of):
            rows = self.place(b, past + m)
            homes = rows[::self.block] // self.block
            for i, home in enumerate(homes.tolist()):
                want, step = BR.bounds_of(k[rows[i * self.block:(i + 1) * self.block]])
                assert torch.equal(bounds[home], want) and torch.equal(steps[home], step), (b, i)
            for i in sorted({0, m // 2, m - 1}) if m else []:
                n, t = past + i + 1, at + i
                nb = -(-n // self.block)
                for g in range(self.hkv):
                    h = slice(g * grp, (g + 1) * grp)
                    s = BR.scores(BR.whole(query[t, h]), bounds[homes[:nb], g], steps[homes[:nb], g])
                    sel = BR.pick(s, nb, self.nsel, 1, 1)
                    assert blocks[t, g].tolist() == sel + [-1] * (self.nsel - len(sel))
                    tok = torch.cat([torch.arange(x * self.block, min(n, (x + 1) * self.block)) for x in sel])
                    assert int(length[t, g]) == len(tok)
                    for kind, r in ((0, rows[tok]), (1, rows[:n]), (2, rows[:n])):
                        ref, rl, tol, ltol = R.attend(query[t:t + 1, h], k[r, g:g + 1], v[r, g:g + 1], [len(r) - 1],
                                                      self.scale)
                        assert bool(((out[kind][t, h] - ref[0]).abs() <= tol[0]).all()), (b, i, g, kind)
                        assert bool(((lse[kind][t, h] - rl[0]).abs() <= ltol[0]).all()), (b, i, g, kind)
                        # what would not be seen otherwise: zeros, other signs, the values' plain mean
                        for other in (torch.zeros_like(ref[0]), -ref[0]) + ((v[r, g].mean(0),) if len(r) > 1 else ()):
                            assert bool(((other - ref[0]).abs() > tol[0]).any(-1).all())


@pytest.mark.parametrize("kw", [dict(), dict(sb=32, block=16), dict(sb=16, block=32, hq=16), dict(d=128, hkv=4)])
def test_steps_against_what_the_cache_holds(kw):
    s = Checked(4, **kw)
    for i, new in enumerate(STEPS):
        old = s.before()
        s.load(new, i)
        s.x[:sum(new)] *= 2.0 ** (i % 3)  # scales grow in some steps and stay in others
        for b, (at, m, past, q) in enumerate(s.rows_of):
            q *= 2.0 ** (i % 3)
            s.k[b][past:] *= 2.0 ** (i % 3)
            s.v[b][past:] *= 2.0 ** (i % 3)
        s.enqueue()
        torch.cuda.synchronize()
        assert int(s.status) == 0
        s.check_writes(old)
        s.check_rest()


def test_drafts_that_are_taken_back_lose_no_page():
    """Pages opened behind the tokens that stay are put back in front of the free list before the next plan, as its
    description asks: after many steps the pages in use are those of the tokens."""
    s = Checked(3, page=16, max_ctx=256, rows=30)
    g = torch.Generator().manual_seed(3)
    length = [0, 0, 0]
    for step in range(25):
        new = [int(torch.randint(1, 10, (1,), generator=g)) for _ in range(3)]
        for b in range(3):
            s.k[b], s.v[b] = s.k[b][:length[b]], s.v[b][:length[b]]
        s.load(new, step)
        s.enqueue()
        torch.cuda.synchronize()
        assert int(s.status) == 0
        s.check_rest()
        keep = [int(torch.randint(0, n + 1, (1,), generator=g)) for n in new]
        table = s.table.cpu()
        back = []
        for b in range(3):
            back += table[b, -(-(length[b] + keep[b]) // 16):-(-(length[b] + new[b]) // 16)].tolist()
            length[b] += keep[b]
        first = int(s.range[0][0]) - len(back)
        s.free[first:first + len(back)] = torch.tensor(back, dtype=torch.int32, device=s.free.device)
        s.range[0][0] = first
        s.cached.copy_(torch.tensor(length, dtype=torch.int32))
        assert first == sum(-(-n // 16) for n in length)
        used = [p for b in range(3) for p in table[b, :-(-length[b] // 16)].tolist()]
        assert sorted(used + s.free[first:].tolist()) == list(range(s.num_pages))

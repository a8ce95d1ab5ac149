"""Bounds of blocks shorter than the cache's scale blocks: a new token that
raises a scale has the scale block's older codes encoded again, in blocks that
hold no new token."""

from __future__ import annotations

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Growing:
    """Sequences over a block-scaled cache; `add` appends tokens (values times `amp`) and bounds their blocks."""

    def __init__(self, B, hkv, d, sb, block, page, max_ctx=512, seed=0):
        self.B, self.hkv, self.d, self.sb, self.block, self.page, self.max_ctx = B, hkv, d, sb, block, page, max_ctx
        self.g = torch.Generator().manual_seed(seed)
        self.rows = B * max_ctx
        self.table = self.base = None
        if page:
            self.table = torch.randperm(self.rows // page, generator=self.g).int().view(B, -1)
        else:
            self.base = [b * max_ctx for b in range(B)]
        self.length = [0] * B
        self.kc, self.vc = [torch.full((self.rows, hkv, d), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.ks, self.vs = [torch.ones(self.rows // sb, hkv, device=DEV) for _ in range(2)]
        self.bounds = torch.full((self.rows // block, hkv, 2, d), 99, dtype=torch.int8, device=DEV)
        self.steps = torch.full((self.rows // block, hkv), 99.0, device=DEV)
        self.shape = dsa.GqaShape(hkv, hkv, d, dsa.DSA_FP8_E4M3_BLOCKSCALE, scale_block=sb)
        self.status = _i32([0])

    def add(self, new, amp=1.0, heads=slice(None), inserts=1):
        """`inserts` > 1: the tokens in that many writes, the bounds once, of all of them."""
        first = list(self.length)
        for part in range(inserts):
            now = [n * (part + 1) // inserts - n * part // inserts for n in new]
            n = sum(now)
            k, v = [torch.randn(n, self.hkv, self.d, generator=self.g) for _ in range(2)]
            k[:, heads] *= amp
            seqs = self.seqs(self.length, now)
            dsa.dsa_kv_block_insert(self.shape, k.bfloat16().to(DEV), v.bfloat16().to(DEV), None, seqs, n, None, 0,
                                    dsa.DSA_ROPE_PAIRS, self.kc, self.vc, self.ks, self.vs, None, d_status=self.status)
            self.length = [p + m for p, m in zip(self.length, now)]
        dsa.block_gqa_bounds(self.shape, self.kc, self.ks, self.seqs(first, new), sum(new), self.block, self.bounds,
                             self.steps, d_status=self.status)
        torch.cuda.synchronize()
        assert int(self.status) == 0

    def seqs(self, past, new):
        q_start = [0]
        for m in new:
            q_start.append(q_start[-1] + m)
        return dsa.Seqs(_i32([p + m for p, m in zip(past, new)]), _i32(q_start),
                        _i32([p + i for p, m in zip(past, new) for i in range(m)]), max_ctx=self.max_ctx,
                        max_q_per_seq=max(new), num_rows=self.rows, page_size=self.page,
                        page_table=None if self.table is None else self.table.to(DEV),
                        seq_base=None if self.base is None else torch.tensor(self.base, device=DEV))

    def check(self):
        """Every block that holds keys has the bounds of the keys that the cache holds now; the others none."""
        scale = self.ks.cpu().repeat_interleave(self.sb, 0)
        keys = (self.kc.cpu().view(torch.float8_e4m3fn).float() * scale[..., None]).double()
        bounds, steps = torch.full_like(self.bounds.cpu(), 99), torch.full_like(self.steps.cpu(), 99.0)
        for b, n in enumerate(self.length):
            rows = R.rows_of(self.table, self.page, self.base, b, n)
            for i in range(0, n, self.block):
                home = int(rows[i]) // self.block
                bounds[home], steps[home] = BR.bounds_of(keys[rows[i:i + self.block]])
        assert torch.equal(self.steps.cpu(), steps)
        assert torch.equal(self.bounds.cpu(), bounds)


@pytest.mark.parametrize("sb, block, page", [(64, 16, 64), (128, 16, 256), (128, 64, 128), (32, 16, 32), (64, 32, 0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [1, 4, 15, 20, 40])
def test_a_token_that_raises_a_scale(sb, block, page, d, power):
    """The older codes lose bits below the smallest normal code: the bounds of all their blocks follow."""
    s = Growing(3, 3, d, sb, block, page, seed=power)
    s.add([sb - 5, sb // 2 + 3, 2 * sb - 1])
    s.check()
    s.add([1, 2, 1], amp=2.0 ** power, heads=slice(1, 2))
    s.check()
    s.add([9, 1, 30], amp=2.0 ** (2 * power), heads=slice(0, 2))
    s.check()


def test_every_token_raises_it():
    """Token by token, each twice the last; then several writes before their bounds."""
    s = Growing(2, 2, 64, 128, 16, 128, seed=1)
    for i in range(100):
        s.add([1, 1], amp=2.0 ** (i / 4 - 10))
    s.check()
    s.add([20, 24], amp=2.0 ** 30, inserts=4)
    s.check()


def test_other_blocks_are_left():
    """Where the new tokens raise no scale, and in other scale blocks, nothing is written."""
    s = Growing(1, 2, 64, 64, 16, 64, seed=2)
    s.add([120])
    s.bounds[:], s.steps[:] = 99, 99.0
    s.add([1], amp=2.0 ** -3)
    touched = (s.steps != 99).any(-1).nonzero().flatten().tolist()
    rows = R.rows_of(s.table, 64, None, 0, 121)
    assert touched == [int(rows[120]) // 16]
    s.steps[:] = 99.0
    s.add([1], amp=2.0 ** 12)  # the second scale block: tokens 64 .. 121
    touched = sorted((s.steps != 99).any(-1).nonzero().flatten().tolist())
    assert touched == sorted(int(rows[i]) // 16 for i in (64, 80, 96, 112))

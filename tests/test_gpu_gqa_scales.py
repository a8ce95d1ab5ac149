"""e4m3 caches whose values' scales lie far apart: keys that hold the weight keep
their bits beside keys with scales up to 2^100 times theirs that hold none, or
whose product with their weight is of the same size."""

from __future__ import annotations

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


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("shift, amp", [(7, 1.0), (24, 4.0), (34, 4.0), (60, 4.0), (60, 1.0), (60, 0.5), (100, 4.0)])
@pytest.mark.parametrize("ctx, new, hq, hkv, d", [([700], [1], 16, 2, 128), ([5000, 70], [1, 1], 8, 8, 64),
                                                  ([3000], [2], 16, 2, 128), ([900, 4000], [4, 3], 16, 2, 128),
                                                  ([900], [4], 16, 2, 64), ([40000], [1], 16, 2, 128),
                                                  ([30000, 25], [3, 1], 16, 2, 64)])
def test_large_scales_of_keys_without_weight(call, shift, amp, ctx, new, hq, hkv, d):
    """Every eighth key of the first 256 and a few behind them: scores some 40 amp below the others'
    (for amp 1 a weight of 2^-58 or so), scales 2^shift times the others'.  Their values are 0 in every other
    dim: there the other keys alone count, however small their products are beside the largest."""
    c = Case(ctx, new, hq, hkv, d, e4m3=True, page=64, seed=shift)
    c.q = (c.q.float().abs() * amp).bfloat16()
    for b, n in enumerate(ctx):
        rows = R.rows_of(c.table, 64, None, b, n)
        at = rows[[j for j in range(n) if (j < 256 and j % 8 == 3) or j % 613 == 600]]
        c.k[at] = 0xFE  # -448
        c.ks[at] = 0.01 if d == 128 else 0.0141
        c.v[at, :, ::2] = 0
        c.vs[rows] *= 2.0 ** (-shift / 2)
        c.vs[at] *= 2.0 ** shift
    c.dq, c.dk, c.dv, c.dks, c.dvs = [x.to(DEV) for x in (c.q, c.k, c.v, c.ks, c.vs)]
    c.run(call).check()


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("new", [1, 2, 4])
def test_scales_of_every_size(call, new):
    """Scales spread evenly over 2^-60 to 2^60, every key of the same weight or nearly so: what counts are the
    largest; and with their scores lowered by as much, all count alike."""
    for lowered in (False, True):
        c = Case([2000], [new], 16, 2, 128, e4m3=True, page=64, seed=new)
        rows = R.rows_of(c.table, 64, None, 0, 2000)
        g = torch.Generator().manual_seed(new)
        p = torch.randint(-60, 61, (2000, 2), generator=g)
        c.vs[rows] = c.vs[rows] * 2.0 ** p.float()
        if lowered:
            # q's first dim 1, the others small; the key's first value -p ln 2 / scale, as a code near it
            c.q = (c.q.float() * 0.05).bfloat16()
            c.q[..., 0] = 1.0
            c.ks[rows] = 0.125
            want = (-p.float() * 0.6931 / (0.125 * c.sm_scale)).clamp(-448, 448)
            c.k[rows, :, 0] = want.to(torch.float8_e4m3fn).view(torch.uint8)
        c.dq, c.dk, c.dks, c.dvs = [x.to(DEV) for x in (c.q, c.k, c.ks, c.vs)]
        c.run(call).check()

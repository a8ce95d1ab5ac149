"""Dense grouped-head attention over contexts of millions of tokens, whose pages
are one page: the result is the attention over that page's rows, the last
page's counted as far as they are seen."""

from __future__ import annotations

import math

import pytest
import torch

import dsa_sparse_mla_query_gb300 as dsa
import gqa_reference as R
from test_gpu_gqa import CALLS, DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ctx", [(1 << 22) - 3, (1 << 22) + 77, (1 << 24) + 1])
def test_contexts_of_millions(call, e4m3, ctx):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    page, hq, hkv, d, new = 256, 4, 2, 64, 5
    g = torch.Generator().manual_seed(ctx % 1000)
    q = torch.randn(new, hq, d, generator=g).bfloat16()
    if e4m3:
        k, v = [(torch.randn(page, hkv, d, generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for _ in range(2)]
        ks, vs = [torch.rand(page, hkv, generator=g) * 0.01 + 0.002 for _ in range(2)]
    else:
        k, v = [torch.randn(page, hkv, d, generator=g).bfloat16() for _ in range(2)]
        ks = vs = None
    i32 = dict(dtype=torch.int32, device=DEV)
    pos = [ctx - 1, 5, ctx - 200, 1 << 21, ctx // 2]
    dev = lambda x: None if x is None else x.to(DEV)
    dk, dv, dks, dvs = dev(k), dev(v), dev(ks), dev(vs)
    seqs = dsa.Seqs(torch.tensor([ctx], **i32), torch.tensor([0, new], **i32), torch.tensor(pos, **i32), max_ctx=ctx,
                    max_q_per_seq=new, num_rows=page, page_table=torch.zeros(1, (ctx + page - 1) // page, **i32),
                    page_size=page)
    shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16)
    nb = dsa.dense_gqa_workspace_size(shape, seqs, new)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    out, lse = torch.full((new, hq, d), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((new, hq), 7.0, device=DEV)
    status = torch.zeros(1, **i32)
    scale = 1 / math.sqrt(d)
    CALLS[call](shape, q.to(DEV), dk, dv, dks, dvs, seqs, new, scale, out, lse, ws, nb, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    kk, vv = R.values(k, ks), R.values(v, vs)
    for t, p in enumerate(pos):
        times = torch.tensor([(p + 1) // page + (r < (p + 1) % page) for r in range(page)], dtype=torch.float64)
        for h in range(hq):
            s = scale * (kk[:, h // 2] @ q[t, h].double())
            top = torch.logsumexp(s + torch.log(times), 0)
            w = torch.exp(s - top) * times
            ref, av = w @ vv[:, h // 2], w @ vv[:, h // 2].abs()
            # half a step of the result and of every weight; sums of n / 16 fp32 additions; scores (sums
            # of 64 products, below 64) off by 2^-24 of some hundred
            adds = 2.0 ** -24 * (p / 16 + 64)
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * adds + 2.0 ** -15) * av
            assert bool(((out[t, h].double().cpu() - ref).abs() <= tol).all()), (t, h)
            assert abs(float(lse[t, h]) - float(top)) <= adds + 2.0 ** -15

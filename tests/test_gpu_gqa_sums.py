"""Dense grouped-head attention: sums of very many small weights beside a large
one, each of which a running fp32 sum would lose."""

from __future__ import annotations

import math

import pytest
import torch

import dsa_sparse_mla_query_gb300 as dsa
from test_gpu_gqa import CALLS, DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_weights_below_half_a_step(call, e4m3):
    """The first key's weight is 1, the 65,535 others' e^-16.75, 0.89 of half a step of 1.  Every score is one
    exact product.  Allowed: chains of n / 16 + 64 additions, each off by half a step of the sum; the weights'
    own errors (scores of 16.75 off by a few steps, 2^-18 of a weight) are 2^-18 of all of them together."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    n, new, hq, d = 65536, 1300, 64, 64
    k = torch.zeros(n, 1, d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[1:, 0, 0] = 0xD8 if e4m3 else -16.75  # -16, the scale 1.046875
    scale = torch.full((n, 1), 1.046875, device=DEV) if e4m3 else None
    q = torch.zeros(new, hq, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    i32 = dict(dtype=torch.int32, device=DEV)
    pos = n - 1 - torch.arange(new, **i32) % 7
    seqs = dsa.Seqs(torch.tensor([n], **i32), torch.tensor([0, new], **i32), pos, max_ctx=n, max_q_per_seq=new,
                    num_rows=n, seq_base=torch.zeros(1, dtype=torch.int64, device=DEV))
    shape = dsa.GqaShape(hq, 1, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16)
    nb = dsa.dense_gqa_workspace_size(shape, seqs, new)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(new, hq, device=DEV)
    status = torch.zeros(1, **i32)
    CALLS[call](shape, q, k, v, scale, scale, seqs, new, 1.0, out, lse, ws, nb, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = torch.log1p(pos.double() * math.exp(-16.75)).cpu()[:, None]
    rest = n * math.exp(-16.75)
    tol = (n / 16 + 64) * 2.0 ** -24 * (1 + rest) + 2.0 ** -18 * rest + 8 * 2.0 ** -24
    assert float((lse.double().cpu() - want).abs().max()) <= tol

"""Paths of the block selection and of attention over listed blocks that long
batches take: many sequences beside a prompt, whole lists in turn with tiles of
16 and 32 query rows, malformed sequences call by call."""

from __future__ import annotations

import math

import pytest
import torch

import block_reference as BR
import dsa_sparse_mla_query_gb300 as dsa
from test_gpu_block_select import BAD, DEV, KINDS, Step, _few, _i32, _random_lists

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    dsa.load()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# many sequences, one of them a prompt: the scores of every sequence by the tensor cores' kernel
def _mixed(n, prompt, at, *, step=3, hq=8, hkv=2, d=64, page=16, **kw):
    """`n` sequences, most with one token or none, number `at` with `prompt` of them."""
    new = [prompt if b == at else int(b % step == 0) for b in range(n)]
    ctx = [prompt + 70 if b == at else 1 + b % 90 for b in range(n)]
    return Step(ctx, new, hq, hkv, d, 16, kv="bf16", page=page, nsel=5, first=1, local=2, seed=n, extra_q=3, **kw)


@pytest.mark.parametrize("n, at", [(33, 32), (40, 0), (100, 57), (2177, 2176), (2300, 2200), (4400, 4399)])
def test_select_of_a_prompt_among_many_sequences(n, at):
    s = _mixed(n, 300, at, step=50 if n > 1000 else 3).run_select()
    some = _few(s, 25) or list(range(s.nq))
    start = s.q_start[at]
    s.check_select(sorted(set(some) | {start, start + 150, start + 299}))


@pytest.mark.parametrize("n", [1025, 2100])
def test_bounds_of_more_sequences_than_a_scan_holds(n):
    """1,024 at a time."""
    _mixed(n, 40, n - 2).run_bounds().check_bounds()


def test_a_mixed_step():
    """A prompt's chunk beside decoding sequences: bounds, selection, attention."""
    s = _mixed(50, 300, 20, d=128, hq=16).run_bounds().run_select().run_attend()
    s.check_select(_few(s))
    s.check_attend(_few(s))


# ---------------------------------------------------------------------------
# whole lists in turn (eight lists or more a CTA), tiles of 16 and 32 rows, two chunks of heads
@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("hq, hkv, d, tokens", [(32, 2, 128, 650), (32, 2, 64, 650), (40, 2, 64, 620), (33, 1, 128, 640),
                                                (64, 1, 64, 1300), (9, 1, 128, 1300)])
def test_whole_lists_in_turn_with_many_rows(kv, hq, hkv, d, tokens):
    s = Step([tokens + 60], [tokens], hq, hkv, d, 32, kv=kv, page=32, nsel=4, seed=hq, extra_q=1)
    _random_lists(s, seed=tokens)
    s.run_attend().check_attend(_few(s, 12))


# ---------------------------------------------------------------------------
# malformed sequences
def _shapes():
    """Few rows a sequence; many, so that the tensor cores score them and a warp chooses a row."""
    yield "few", dict(ctx=[900, 500, 64], new=[2, 2, 1], hq=8, hkv=2)
    yield "wide", dict(ctx=[900, 500, 1400], new=[2, 2, 1300], hq=8, hkv=4)


SHAPES = dict(_shapes())


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("what", ["a negative context", "a context past max_ctx", "more rows than max_q_per_seq"])
def test_a_malformed_sequence_alone_is_left(name, what):
    """Each call reports it, and the other sequences have what they would have without it."""
    a = SHAPES[name]
    s = Step(a["ctx"], a["new"], a["hq"], a["hkv"], 64, 32, page=32, seed=4)
    bad = 1
    if what == "more rows than max_q_per_seq":
        bad = 2 if name == "wide" else 0
        if name == "few":
            s.seqs.max_q_per_seq = 1  # of two tokens: sequences 0 and 1
    ctx = list(a["ctx"])
    if what == "a negative context":
        ctx[bad] = -1
    elif what == "a context past max_ctx":
        ctx[bad] = max(a["ctx"]) + 1
    elif name == "wide":
        s.seqs.max_q_per_seq = 1299
    s.seqs.ctx_len = _i32(ctx)
    lost = {0, 1} if what == "more rows than max_q_per_seq" and name == "few" else {bad}
    rows = [t for t in range(s.nq) if s.seq[t] not in lost]
    gone = [t for t in range(s.nq) if s.seq[t] in lost]
    some = rows[::max(1, len(rows) // 12)]

    def fresh():
        torch.cuda.synchronize()
        s.status.zero_()

    s.run_bounds().check_bounds(skip=lost, status=BAD)
    fresh()
    s.run_select().check_select(some, status=BAD)
    assert bool((s.blocks[gone] == 77).all()) and bool((s.len[gone] == 77).all())
    fresh()
    # listed attention: the malformed sequence's keys and values count as zeros
    s.blocks[gone], s.len[gone] = -1, 5
    s.blocks[gone, :, 0] = 0
    s.run_attend().check_attend(some, status=BAD)
    assert bool((s.out[gone] == 0).all())
    assert bool(((s.lse[gone] - math.log(5)).abs() < 1e-6).all())
    fresh()
    # empty lists read no keys, and the sequence is as malformed
    s.blocks[gone], s.len[gone] = -1, 0
    s.run_attend().check_attend(some, status=BAD)
    assert bool((s.out[gone] == 0).all()) and bool((s.lse[gone] == -math.inf).all())


@pytest.mark.parametrize("n, at", [(3, 0), (40, 1), (2300, 5)])
def test_a_malformed_sequence_without_rows_is_reported(n, at):
    """Behind a prompt that fills the first places of the tensor cores' kernel: the last sequence's context."""
    s = _mixed(n, 300, at, step=50)
    assert s.new[-1] == 0
    ctx = list(s.ctx)
    ctx[-1] = -1
    s.seqs.ctx_len = _i32(ctx)
    s.run_select()
    s.check_select(_few(s, 12), status=BAD)
    s.status.zero_()
    s.run_bounds().check_bounds(status=BAD)


# ---------------------------------------------------------------------------
# the score
@pytest.mark.parametrize("lo, hi", [(-126, 123), (116, 123), (-126, -119)])
@pytest.mark.parametrize("n, ctx, new", [(1, 16 * 300, 1), (1, 16 * 300, 700), (1, 16 * 100, 200), (1, 16 * 3000, 2),
                                         (80, 16 * 100, 1)])
def test_scores_with_every_step_that_bounds_have(n, ctx, new, lo, hi):
    """2^-126 to 2^122 (of the largest fp32 values): the order is that of the exact scores."""
    s = Step([ctx] * n, [new] * n, 4, 4, 128, 16, kv="bf16", page=16, nsel=30, first=1, seed=5)
    g = torch.Generator().manual_seed(2)
    s.steps[:] = torch.exp2(torch.randint(lo, hi, s.steps.shape, generator=g).double()).float()
    s.device()
    s.run_select().check_select(_few(s, 8))


@pytest.mark.parametrize("large", [1.0, 300.0])
def test_how_far_the_score_may_lie_below_a_querys(large):
    """The score bounds q' . k for q' = q in whole steps; |q - q'| is at most half a step in every dim, so that
    q . k <= step_q score + step_q / 2 sum_d |k_d|, with a few dims far above the others as well."""
    s = Step([512], [512], 8, 2, 64, 16, kv="bf16", page=64, seed=3)
    s.q[:, :, 5] *= large
    s.device()
    s.run_bounds()
    assert s.stat() == 0
    rows = s.rows_of(0)
    k = s.values("k")[rows]
    home = torch.tensor([int(rows[i * 16]) // 16 for i in range(32)])
    for t in range(0, 512, 37):
        for g in range(2):
            q = s.q[t, 4 * g:4 * g + 4].double()
            step = BR.step_of(float(q.abs().max()))
            score = step * BR.scores(BR.whole(q), s.dbounds.cpu()[home, g], s.dsteps.cpu()[home, g])
            slack = step / 2 * k[:, g].abs().sum(-1)
            best = ((q @ k[:, g].T) - slack).amax(0).view(32, 16).amax(1)
            assert bool((score >= best - 1e-9 * best.abs()).all())


# ---------------------------------------------------------------------------
# layouts
@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("new", [1, 600])
def test_keys_and_values_in_one_cache(kv, new):
    """Rows [keys' heads, values' heads, something else] of one buffer, for the three calls."""
    s = Step([700, 90], [new, 1], 8, 2, 128, 32, kv=kv, page=64, nsel=5, first=1, local=2, seed=new)
    both = torch.zeros(s.rows, 5, 128, dtype=s.dk.dtype, device=DEV)
    if kv == "bf16":
        both[:, 4] = math.nan
    else:
        both[:, 4] = 0x7F
    both[:, :2], both[:, 2:4] = s.dk, s.dv
    s.dk, s.dv = both[:, :2], both[:, 2:]
    s.shape = dsa.GqaShape(8, 2, 128, KINDS[kv], q_stride=s.dq.stride(0), k_stride=5 * 128, v_stride=5 * 128,
                           scale_block=s.sb if kv == "block" else 0)
    s.run_bounds().check_bounds()
    s.run_select().run_attend()
    s.check_select(_few(s, 12))
    s.check_attend(_few(s, 12))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("block, ctx", [(64, 500), (16, 500), (128, 259)])
@pytest.mark.parametrize("new", [1, 200])
def test_a_cache_that_ends_inside_a_block(kv, block, ctx, new):
    """Contiguous rows up to the cache's last one; bounds and scales of the last block are there, its other rows not."""
    s = Step([ctx], [new], 16, 2, 64, block, kv=kv, sb=64 if kv == "block" else 0, nsel=3, seed=ctx)
    s.seqs.num_rows = ctx
    s.dk, s.dv = s.dk[:ctx].clone(), s.dv[:ctx].clone()
    if kv == "row":
        s.dks, s.dvs = s.dks[:ctx].clone(), s.dvs[:ctx].clone()
    elif kv == "block":
        s.dks, s.dvs = [x[:-(-ctx // 64)].clone() for x in (s.dks, s.dvs)]
    n = -(-ctx // block)
    left = s.dbounds[n:].clone(), s.dsteps[n:].clone()
    s.run_bounds().check_bounds()
    assert torch.equal(left[0], s.dbounds[n:]) and torch.equal(left[1], s.dsteps[n:])
    s.run_select().run_attend()
    s.check_select(_few(s, 12))
    s.check_attend(_few(s, 12))


@pytest.mark.parametrize("d, half", [(64, False), (128, True)])
def test_writes_and_dense_calls_over_one_cache_that_ends_inside_a_block(d, half):
    """The same bits as with a cache for keys and one for values, each whole blocks."""
    hq, hkv, sb, rows, past, new = 8, 2, 64, 250, 70, 180
    g = torch.Generator().manual_seed(d)
    x = torch.randn(new, hq + 2 * hkv, d, generator=g).bfloat16().to(DEV)
    code = torch.randint(0, 0x70, (256, 5, d), generator=g).to(torch.uint8).to(DEV)
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    got = []
    for shared in (False, True):
        both = code[:rows].clone() if shared else code.clone()
        if shared:
            k, v = both[:, :2], both[:, 2:4]
            stride = 5 * d
        else:
            k, v, stride = both[:, :2].contiguous(), both[:, 2:4].contiguous(), 0
        ks, vs = [torch.full((4, hkv), 2.0 ** -7, device=DEV) for _ in range(2)]
        shape = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_BLOCKSCALE, k_stride=stride, v_stride=stride, scale_block=sb)
        seqs = dsa.Seqs(_i32([past + new]), _i32([0, new]), _i32(list(range(past, past + new))), max_ctx=past + new,
                        max_q_per_seq=new, num_rows=rows if shared else 256, seq_base=torch.zeros(1, dtype=torch.int64, device=DEV))
        status, q = _i32([0]), torch.empty(new, hq, d, dtype=torch.bfloat16, device=DEV)
        xq, xk, xv = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        dsa.dsa_kv_block_insert(shape, xk, xv, xq, seqs, new, inv, d, int(half), k, v, ks, vs, q, k_stride=xk.stride(0),
                                v_stride=xv.stride(0), q_stride=xq.stride(0), d_status=status)
        res = [k[:rows].clone(), v[:rows].clone(), ks, vs, q]
        n = dsa.dense_gqa_workspace_size(shape, seqs, new)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        for call in (dsa.dense_gqa_decode, dsa.dense_gqa_prefill):
            out, lse = torch.empty_like(q), torch.empty(new, hq, device=DEV)
            call(shape, q, k, v, ks, vs, seqs, new, 0.1, out, lse, ws, n, d_status=status)
            torch.cuda.synchronize()
            res += [out, lse]
        assert int(status) == 0
        if shared:
            assert torch.equal(both[:, 4], code[:rows, 4])
        got.append(res)
    for a, b in zip(*got):
        assert torch.equal(a, b)

"""A serving step over an 8-bit cache with a scale for each block of tokens and
head, dense or over blocks that a cheap score selects: what is measured.

- plan     dsa_step_plan: page tables, positions and cache slots of a step's
           tokens from the requests' lengths;
- insert   dsa_kv_block_insert: new tokens' keys and values into the cache, a
           power-of-two scale per block of tokens and head, older codes of a
           block encoded again where its scale grows;
- decode   dense_gqa_decode over that cache;
- prompt   dense_gqa_prefill over it (a chunk behind the tokens that it holds);
- select   block_gqa_bounds and block_gqa_select: the bounds of the keys in the
           blocks that new tokens touch, then the best blocks of every query and
           key head by an upper bound of their scores;
- attend   block_gqa_attend: attention over selected blocks.

A case is a dict of plain values; ``prepare`` makes its tensors on the GPU,
``run`` is one pass, in elementary torch operations or (``own``) through the
library, ``exact`` the same outputs in 64 bits from the definition.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -60  # a block of zeros


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # a decode step of 64 sequences, a token each: the step's smallest call, all latency
        dict(name="plan 64x1", op="plan", b=64, past0=32768, past1=32768, new0=1, new1=1, page=64, spare=0),
        # a thousand requests, fresh prompts and running ones, into a graph's fixed number of rows
        dict(name="plan 1000 ragged", op="plan", b=1000, past0=0, past1=4099, new0=1, new1=251, page=64, spare=517),
        # the cache write of that decode step
        dict(name="insert 64x1", op="insert", b=64, past0=32768, past1=32831, new0=1, new1=1, hq=64, hkv=8, d=128,
             sb=64, page=64, rot=64, half=False, fused=True),
        # packed prompts of different lengths, some behind cached tokens
        dict(name="insert 24 prompts", op="insert", b=24, past0=0, past1=4111, new0=17, new1=4095, hq=64, hkv=8,
             d=128, sb=64, page=64, rot=128, half=True, fused=True),
        # decode of a batch of very different contexts, drafts of four tokens to verify
        dict(name="decode 48x4 ragged", op="decode", b=48, past0=57, past1=32763, new0=4, new1=4, hq=64, hkv=8,
             d=128, kv="block", sb=64, page=64),
        # a chunk of a prompt over the cache that holds the tokens before it
        dict(name="prompt chunk 1024 of 32768", op="prompt", b=1, past0=31744, past1=31744, new0=1024, new1=1024,
             hq=64, hkv=8, d=128, kv="block", sb=64, page=64),
        # block selection of a decode step
        dict(name="select 64x32768", op="select", b=64, past0=32767, past1=32767, new0=1, new1=1, hq=64, hkv=8,
             d=128, kv="block", sb=64, page=64, block=64, nsel=32, first=1, local=2),
        # a few very long contexts
        dict(name="select 3x524288", op="select", b=3, past0=524000, past1=524287, new0=1, new1=1, hq=64, hkv=8,
             d=128, kv="bf16", sb=0, page=64, block=64, nsel=64, first=1, local=2),
        # a prompt's chunk: every token selects for itself
        dict(name="select chunk 2048 of 65536", op="select", b=1, past0=63488, past1=63488, new0=2048, new1=2048,
             hq=64, hkv=8, d=128, kv="block", sb=64, page=64, block=64, nsel=32, first=1, local=2),
        # one user, one token: the smallest attention over selected blocks
        dict(name="attend 1x131072 bf16", op="attend", b=1, past0=131071, past1=131071, new0=1, new1=1, hq=64, hkv=8,
             d=128, kv="bf16", sb=0, page=64, block=64, nsel=32, first=1, local=2),
        # attention of the decode step above
        dict(name="attend 64x32768", op="attend", b=64, past0=32767, past1=32767, new0=1, new1=1, hq=64, hkv=8,
             d=128, kv="block", sb=64, page=64, block=64, nsel=32, first=1, local=2),
        # and of the prompt's chunk
        dict(name="attend chunk 2048 of 65536", op="attend", b=1, past0=63488, past1=63488, new0=2048, new1=2048,
             hq=64, hkv=8, d=128, kv="block", sb=64, page=64, block=64, nsel=32, first=1, local=2),
    ]


HEADS = [(64, 8), (32, 4), (32, 32), (16, 2), (12, 4), (40, 8), (8, 1), (5, 5), (14, 2), (32, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "insert", "decode", "prompt", "select", "attend", "attend"])
    page = rng.choice([16, 64, 64, 128, 256])
    if op == "plan":
        b = _log(rng, 1, 4096)
        new1 = max(1, min(_log(rng, 1, 8192), 131072 // b))
        past1 = rng.choice([0, _log(rng, 1, 32768)])
        return dict(op=op, b=b, past0=rng.choice([0, past1 // 2, past1]), past1=past1, new0=rng.choice([0, 1, new1]),
                    new1=new1, page=page, spare=rng.choice([0, _log(rng, 1, 1000)]))
    hq, hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    c = dict(op=op, hq=hq, hkv=hkv, d=d, page=page)
    sb = rng.choice([x for x in (16, 32, 64, 128) if x <= page])
    past1 = _log(rng, 16, 131072)
    if op == "insert":
        b, new1 = _log(rng, 1, 256), _log(rng, 1, 8192)
        past1 = rng.choice([0, min(past1, 8192)])
        while b * (new1 + past1 // 4) * (hq + 2 * hkv) * d > 49000 * 80 * 128:
            b, new1 = (b + 1) // 2, (new1 * 3 + 3) // 4
            past1 = past1 * 3 // 4
        return dict(c, b=b, past0=rng.choice([0, past1]), past1=past1, new0=rng.choice([1, new1]), new1=new1, sb=sb,
                    rot=rng.choice([0, 16, 32, d // 2, d, d]), half=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "decode":
        b, t = _log(rng, 1, 128), rng.choice([1, 1, 2, 4])
        while b * past1 * hkv * d > 48 * 16384 * 8 * 128:
            b, past1 = (b + 1) // 2, max(8, past1 * 3 // 4)
        return dict(c, b=b, past0=rng.choice([0, past1 // 2, past1]), past1=past1, new0=t, new1=t, kv="block", sb=sb)
    if op == "prompt":
        b, new1 = _log(rng, 1, 16), _log(rng, 2, 4096)
        past1 = rng.choice([0, past1])
        while b * new1 * (new1 + past1) * hq * d > 1024 * 32768 * 64 * 128 or b * (new1 + past1) > 131072:
            b, new1, past1 = (b + 1) // 2, (new1 * 3 + 3) // 4, past1 * 3 // 4
        return dict(c, b=b, past0=rng.choice([0, past1]), past1=past1, new0=rng.choice([1, new1]), new1=new1,
                    kv="block", sb=sb)
    kv = rng.choice(["block", "block", "row", "bf16"])
    block = rng.choice([x for x in (16, 32, 64, 128) if x <= page])
    nsel = _log(rng, 4, 64)
    b, new1 = rng.choice([(_log(rng, 1, 128), 1), (_log(rng, 1, 32), 4), (1, _log(rng, 16, 2048))])
    while b * past1 * hkv * d > 48 * 32768 * 8 * 128 or b * new1 * past1 * hq // block > 2048 * 65536 * 64 // 64:
        b, past1 = (b + 1) // 2, max(8, past1 * 3 // 4)
    while b * new1 * hq * nsel * block * d > 2048 * 64 * 2048 * 128 // 2:
        nsel = max(4, nsel // 2)
        new1 = max(1, new1 // 2)
    return dict(c, b=b, past0=rng.choice([0, past1 // 2, past1]), past1=past1, new0=rng.choice([1, new1]), new1=new1,
                kv=kv, sb=sb if kv == "block" else 0, block=block, nsel=nsel, first=rng.choice([0, 1]),
                local=rng.choice([1, 2, 3]))


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread (the longest first)."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(c):
    """(tokens in the cache, new tokens) of each sequence: long pasts meet long and short news."""
    past, new = _spread(c["past0"], c["past1"], c["b"]), _spread(c["new0"], c["new1"], c["b"])
    return past, new[::2] + new[1::2][::-1]


def _token_bytes(c):
    """A token's keys and values in the cache."""
    scale = {"bf16": 0.0, "row": 4.0, "block": 4.0 / max(1, c["sb"])}[c["kv"]]
    return 2 * c["hkv"] * (c["d"] * (2 if c["kv"] == "bf16" else 1) + scale)


def _selected(c, pos):
    """Blocks that a query at `pos` selects, and the keys that it sees in them."""
    have = pos // c["block"] + 1
    n = min(c["nsel"], have)
    return n, (n - 1) * c["block"] + pos % c["block"] + 1


def work(c):
    past, new = _lengths(c)
    nq = sum(new)
    if c["op"] == "plan":
        pages = sum(-(-(p + n) // c["page"]) - -(-p // c["page"]) for p, n in zip(past, new))
        return {"bytes": c["b"] * 16 + (nq + c["spare"]) * 12 + pages * 8, "flops": 2 * nq}
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "insert":
        blocks = sum((p + n - 1) // c["sb"] - p // c["sb"] + 1 for p, n in zip(past, new) if n)
        return {"bytes": nq * (2 * hkv * d * 3 + hq * d * 4 + 4) + blocks * hkv * 8,
                "flops": 3 * nq * c["rot"] * (hq + hkv)}
    if c["op"] in ("decode", "prompt"):
        pairs = sum(m * p + m * (m + 1) // 2 for p, m in zip(past, new))
        return {"bytes": sum(p + m for p, m in zip(past, new)) * _token_bytes(c) + nq * hq * (4 * d + 4),
                "flops": 4 * d * hq * pairs}
    blk = c["block"]
    if c["op"] == "select":
        have = sum(-(-(p + m) // blk) for p, m in zip(past, new))
        rated = sum((p + i) // blk + 1 for p, m in zip(past, new) for i in range(m))
        touched = sum((p + m - 1) // blk - p // blk + 1 for p, m in zip(past, new) if m)
        key = d * (2 if c["kv"] == "bf16" else 1) + {"bf16": 0, "row": 4, "block": 4 / max(1, c["sb"])}[c["kv"]]
        return {"bytes": have * hkv * (2 * d + 4) + touched * hkv * (blk * key + 2 * d + 4) + nq * hq * d * 2
                + nq * hkv * 4 * (c["nsel"] + 1), "flops": 4 * d * hq * rated}
    keys = sum(_selected(c, p + i)[1] for p, m in zip(past, new) for i in range(m))
    # tokens of one sequence may share what they read: at least the longest one's keys, at most the cache
    least = sum(_selected(c, p + m - 1)[1] for p, m in zip(past, new) if m)
    return {"bytes": least * _token_bytes(c) + nq * hq * (4 * d + 4) + nq * hkv * 4 * (c["nsel"] + 1),
            "flops": 4 * d * hq * keys}


# ---------------------------------------------------------------------------
# inputs
def _normal(gen, *shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=gen)


def _codes(gen, *shape):
    """e4m3 codes of normal values, the largest of a block near 448."""
    x = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):  # a piece at a time: the fp32 values are four times the codes
        part = torch.empty(min(1 << 28, flat.numel() - i), dtype=torch.float32, device=DEV).normal_(generator=gen)
        flat[i:i + part.numel()] = (part * 90.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _cache(c, gen, rows, values):
    """k, v [rows, hkv, d] and their scales ([rows, hkv] or [rows / sb, hkv], powers of two there)."""
    hkv, d = c["hkv"], c["d"]
    if c["kv"] == "bf16":
        return _normal(gen, rows, hkv, d), _normal(gen, rows, hkv, d) if values else None, None, None
    k, v = _codes(gen, rows, hkv, d), _codes(gen, rows, hkv, d) if values else None

    def scales():
        if c["kv"] == "row":
            return torch.rand(rows, hkv, generator=gen, device=DEV) * 0.004 + 0.004
        return _two_to(torch.randint(-8, -5, (rows // c["sb"], hkv), generator=gen, device=DEV))

    return k, v, scales(), scales() if values else None


def _tokens(gen, n, hq, hkv, d, fused):
    """q, k, v [n, heads, d] of new tokens: slices of one projection, or tensors of their own."""
    if fused:
        x = _normal(gen, n, hq + 2 * hkv, d)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return _normal(gen, n, hq, d), _normal(gen, n, hkv, d), _normal(gen, n, hkv, d)


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def _lists(c, s, gen):
    """Selected blocks [nq, hkv, nsel] (ascending, -1 behind them) and the keys seen [nq, hkv]: the first
    and the nearest blocks, the others those that neighbouring tokens mostly share."""
    blk, nsel, hkv, nq = c["block"], c["nsel"], c["hkv"], s["nq"]
    out = torch.full((nq, hkv, nsel), -1, dtype=torch.int32, device=DEV)
    at = 0
    for p, m in zip(*s["lens"]):
        width = (p + m - 1) // blk + 1
        for i in range(0, m, 64):
            e = min(m, i + 64)
            pos = torch.arange(p + i, p + e, device=DEV)
            rank = torch.rand(1, hkv, width, generator=gen, device=DEV) \
                + 0.2 * torch.rand(e - i, hkv, width, generator=gen, device=DEV)
            j = torch.arange(width, device=DEV)
            own_block = (pos // blk)[:, None]
            near = (j > own_block - c["local"]) & (j <= own_block)
            rank[(near | (j < c["first"]))[:, None].expand_as(rank)] += 4.0
            rank[near[:, None].expand_as(rank)] += 4.0  # the own block stays where there are few
            rank[(j > own_block)[:, None].expand_as(rank)] = -1.0
            n = min(nsel, width)
            v, idx = rank.topk(n, -1)
            idx = torch.where(v < 0, torch.full_like(idx, 1 << 30), idx).sort(-1).values
            out[at + i:at + e, :, :n] = torch.where(idx == 1 << 30, torch.full_like(idx, -1), idx).int()
        at += m
    pos = s["q_pos"].long()
    n = torch.clamp(pos // blk + 1, max=nsel)
    return out, ((n - 1) * blk + pos % blk + 1).int()[:, None].expand(nq, hkv).contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    past, new = _lengths(c)
    order = rng.permutation(c["b"])
    past, new = [past[i] for i in order], [new[i] for i in order]
    page, nq = c["page"], sum(new)
    ctx = [p + n for p, n in zip(past, new)]
    had, used = [-(-p // page) for p in past], [-(-x // page) for x in ctx]
    width = max(1, max(used)) + 1
    pages = rng.permutation(sum(used) + 9)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device=DEV), lens=(past, new), nq=nq,
             num_pages=len(pages))
    table = np.full((c["b"], width), -1, np.int32)
    at = 0
    for i in range(c["b"]):
        fill = had[i] if c["op"] == "plan" else used[i]
        table[i, :fill] = pages[at:at + fill]
        at += fill
    s["page_table"] = _i32(table)
    if c["op"] == "plan":
        s["cached"], s["new"] = _i32(past), _i32(new)
        s["free"] = _i32(pages[at:])
        s["free_range"] = _i32([2, len(pages) - at])  # two pages were taken before
        s["rows"] = nq + c["spare"]
        for name, shape, t in (("ctx", c["b"], torch.int32), ("q_start", c["b"] + 1, torch.int32),
                               ("q_pos", s["rows"], torch.int32), ("slot", s["rows"], torch.int64),
                               ("next", 2, torch.int32)):
            s[name] = torch.zeros(shape, dtype=t, device=DEV)
        return s

    q_start = np.concatenate([[0], np.cumsum(new)])
    rows = len(pages) * page
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    s.update(rows=rows, ctx=_i32(ctx), q_start=_i32(q_start), max_ctx=max(ctx), max_new=max(new),
             q_pos=_i32(np.concatenate([np.arange(p, x) for p, x in zip(past, ctx)])), sm_scale=1.0 / math.sqrt(d))
    if own:
        import dsa_sparse_mla_query_gb300 as dsa
        s["seqs"] = dsa.Seqs(s["ctx"], s["q_start"], s["q_pos"], max_ctx=s["max_ctx"], max_q_per_seq=s["max_new"],
                             num_rows=rows, page_table=s["page_table"], page_size=page)
        kinds = {"bf16": dsa.DSA_BF16, "row": dsa.DSA_FP8_E4M3_ROWSCALE, "block": dsa.DSA_FP8_E4M3_BLOCKSCALE}
        s["shape"] = dsa.GqaShape(hq, hkv, d, kinds[c.get("kv", "block")], scale_block=c["sb"])
    if c["op"] == "insert":
        c = dict(c, kv="block")
        s["q"], s["k"], s["v"] = _tokens(gen, nq, hq, hkv, d, c["fused"])
        s["inv_freq"] = None
        if c["rot"]:
            i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-i / c["rot"])).float().to(DEV)
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(c, gen, rows, True)
        s["q_out"] = torch.empty(nq, hq, d, dtype=torch.bfloat16, device=DEV)
        return s
    s["q"] = _normal(gen, nq, hq, d)
    s["k"], s["v"], s["k_scale"], s["v_scale"] = _cache(c, gen, rows, c["op"] != "select")
    if c["op"] == "select":
        # the bounds of 16 to 128 normal keys lie around 2 to 3 deviations: codes of some 50 to 127
        n = rows // c["block"]
        mean = math.sqrt(2 * math.log(c["block"])) * 36
        x = torch.empty(n, hkv, 2, d, dtype=torch.float32, device=DEV).normal_(generator=gen)
        x = (x * 14 + mean).round_().clamp_(-20, 127)
        x[:, :, 0].neg_()
        s["bounds"] = x.to(torch.int8)
        s["bound_scale"] = _two_to(torch.randint(-6, -4, (n, hkv), generator=gen, device=DEV))
        s["blocks"] = torch.empty(nq, hkv, c["nsel"], dtype=torch.int32, device=DEV)
        s["sel_len"] = torch.empty(nq, hkv, dtype=torch.int32, device=DEV)
    else:
        s["out"] = torch.empty(nq, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(nq, hq, dtype=torch.float32, device=DEV)
    if c["op"] == "attend":
        s["blocks"], s["sel_len"] = _lists(c, s, gen)
    if own:
        s["ws_bytes"] = dsa.block_gqa_workspace_size(s["shape"], s["seqs"], nq, c["block"], c["nsel"]) \
            if c["op"] in ("select", "attend") else dsa.dense_gqa_workspace_size(s["shape"], s["seqs"], nq)
        s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan_plain, "insert": _insert_plain, "decode": _dense_plain, "prompt": _dense_plain,
            "select": _select_plain, "attend": _attend_plain}[s["case"]["op"]](s)


def _run_own(s):
    import dsa_sparse_mla_query_gb300 as dsa
    c = s["case"]
    if c["op"] == "plan":
        dsa.dsa_step_plan(s["cached"], s["new"], c["b"], s["free"], s["free_range"], c["page"], s["num_pages"],
                          s["page_table"], s["rows"], s["ctx"], s["q_start"], s["q_pos"], s["slot"], s["next"],
                          d_status=s["status"])
        return _planned(s)
    if c["op"] == "insert":
        q, k, v = s["q"], s["k"], s["v"]
        dsa.dsa_kv_block_insert(s["shape"], k, v, q, s["seqs"], s["nq"], s["inv_freq"], c["rot"],
                                dsa.DSA_ROPE_HALVES if c["half"] else dsa.DSA_ROPE_PAIRS, s["k_cache"], s["v_cache"],
                                s["k_scale"], s["v_scale"], s["q_out"], k_stride=k.stride(0), v_stride=v.stride(0),
                                q_stride=q.stride(0), d_status=s["status"])
        return _inserted(s)
    if c["op"] == "select":
        dsa.block_gqa_bounds(s["shape"], s["k"], s["k_scale"], s["seqs"], s["nq"], c["block"], s["bounds"],
                             s["bound_scale"], d_status=s["status"])
        dsa.block_gqa_select(s["shape"], s["q"], s["bounds"], s["bound_scale"], s["seqs"], s["nq"], c["block"],
                             c["nsel"], c["first"], c["local"], s["blocks"], s["sel_len"], s["ws"], s["ws_bytes"],
                             d_status=s["status"])
        return {n: s[n] for n in ("bounds", "bound_scale", "blocks", "sel_len")}
    if c["op"] == "attend":
        dsa.block_gqa_attend(s["shape"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["seqs"], s["nq"],
                             s["blocks"], s["sel_len"], c["block"], c["nsel"], s["sm_scale"], s["out"], s["lse"],
                             s["ws"], s["ws_bytes"], d_status=s["status"])
    else:
        dense = dsa.dense_gqa_decode if c["op"] == "decode" else dsa.dense_gqa_prefill
        dense(s["shape"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["seqs"], s["nq"], s["sm_scale"],
              s["out"], s["lse"], s["ws"], s["ws_bytes"], d_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _planned(s):
    return {n: s[n] for n in ("page_table", "ctx", "q_start", "q_pos", "slot", "next")}


def _inserted(s):
    """The caches' codes as the e4m3 values that they stand for, their scales and the rotated queries."""
    return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": s["q_out"]}


def _plan_plain(s):
    c = s["case"]
    page, rows = c["page"], s["rows"]
    past, new = s["cached"].long(), s["new"].long()
    ctx = past + new
    start = torch.zeros(c["b"] + 1, dtype=torch.long, device=DEV)
    start[1:] = torch.cumsum(new, 0)
    had = (past + page - 1) // page
    more = (ctx + page - 1) // page - had
    taken = torch.cumsum(more, 0)
    # a row's sequence: the number of sequences that end at or before it
    t = torch.arange(rows, device=DEV)
    live = t < start[-1]
    at = torch.where(live, t, torch.zeros_like(t))  # the rows behind the last do what the first does
    b = torch.searchsorted(start[1:], at, right=True)
    pos = past[b] + at - start[b]
    col = pos // page
    fresh = col >= had[b]
    src = torch.where(fresh, s["free_range"][0] + taken[b] - more[b] + col - had[b], torch.zeros_like(col))
    held = s["page_table"][b, col]
    own_page = torch.where(fresh, s["free"][src.clamp(max=s["free"].numel() - 1)], held).long()
    slot = torch.where(live, own_page * page + pos % page, torch.full_like(pos, -1))
    s["page_table"][b, col] = own_page.int()
    s["ctx"], s["q_start"] = ctx.int(), start.int()
    s["q_pos"] = torch.where(live, pos, torch.full_like(pos, -1)).int()
    s["slot"] = slot
    s["next"] = torch.stack([s["free_range"][0] + taken[-1].int(), s["free_range"][1]])
    return _planned(s)


def _rows(s, b, j):
    """Physical rows of tokens j of sequences b."""
    page = s["case"]["page"]
    return s["page_table"][b, j // page].long() * page + j % page


def _rotate_plain(x, pos, inv_freq, rot, half):
    """x [n, heads, d] in fp32, its first `rot` dims rotated by pos * inv_freq (angles in fp64)."""
    if not rot:
        return x
    ang = pos.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    y = x.clone()
    if half:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _two_to(e):
    """2^e in fp32, e whole numbers in [-126, 127]"""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pow2_above(x):
    """The least power of two not below x > 0 (frexp: x = m 2^e, m in [0.5, 1))."""
    m, e = torch.frexp(x)
    return _two_to(torch.where(m == 0.5, e - 1, e).clamp(min=-126))


def _blocks_of_new(s):
    """(sequence of each new token, its physical block) and whether older tokens share the block."""
    sb = s["case"]["sb"]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=s["nq"])
    pos = s["q_pos"].long()
    row = _rows(s, b, pos)
    older = (s["ctx"].long() - n)[b]                     # the sequence's first new position
    return row, row // sb, torch.clamp(older - pos // sb * sb, min=0)  # older tokens in the token's block


def _store_plain(x, row, blk, older, cache, scale, sb):
    """x [n, hkv, d] in fp32 into the codes [rows, hkv, d] and the scales [rows / sb, hkv]."""
    amax = x.abs().amax(-1)                                                   # [n, hkv]
    top = torch.zeros_like(scale).scatter_reduce(0, blk[:, None].expand_as(amax), amax, "amax")
    need = _pow2_above(torch.clamp(top / E4M3_MAX, min=LEAST_SCALE))
    # (top / 448 rounds, but not across a power of two: 448 2^k / 448 is exact)
    held = torch.zeros(scale.shape[0], dtype=torch.long, device=DEV).scatter_reduce(0, blk, older, "amax")
    fresh = torch.zeros_like(held).scatter(0, blk, 1)
    keep = (held > 0)[:, None]
    now = torch.where((fresh > 0)[:, None], torch.where(keep, torch.maximum(scale, need), need), scale)
    # older codes of blocks whose scale grew
    grown = torch.nonzero((keep & (now > scale)).any(-1))[:, 0]
    old_row = grown[:, None] * sb + torch.arange(sb, device=DEV)
    inside = torch.arange(sb, device=DEV) < held[grown][:, None]
    old_row, of = old_row[inside], grown[:, None].expand_as(inside)[inside]
    old = cache[old_row].view(torch.float8_e4m3fn).float() * (scale[of] / now[of])[..., None]
    cache[old_row] = old.to(torch.float8_e4m3fn).view(torch.uint8)
    cache[row] = (x / now[blk][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(now)


def _insert_plain(s):
    c = s["case"]
    row, blk, older = _blocks_of_new(s)
    k = _rotate_plain(s["k"].float(), s["q_pos"], s["inv_freq"], c["rot"], c["half"])
    _store_plain(k, row, blk, older, s["k_cache"], s["k_scale"], c["sb"])
    _store_plain(s["v"].float(), row, blk, older, s["v_cache"], s["v_scale"], c["sb"])
    s["q_out"] = _rotate_plain(s["q"].float(), s["q_pos"], s["inv_freq"], c["rot"], c["half"]).bfloat16()
    return _inserted(s)


def _gather(s, x, scale, row, h):
    """fp32 values of rows `row` (any shape), head h."""
    c = s["case"]
    if c["kv"] == "bf16":
        return x[row, h].float()
    at = row if c["kv"] == "row" else row // c["sb"]
    return x.view(torch.float8_e4m3fn)[row, h].float() * scale[at, h][..., None]


def _dense_plain(s):
    """Padded to the longest sequence and the most new tokens; one key head at a time bounds the memory."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, b, t, n = hq // hkv, c["b"], s["max_new"], s["max_ctx"]
    j = torch.arange(n, device=DEV)
    i = torch.arange(t, device=DEV)
    row = torch.where(j < s["ctx"][:, None], s["page_table"].long()[:, j // c["page"]] * c["page"] + j % c["page"],
                      torch.zeros(1, dtype=torch.long, device=DEV))                  # [b, n]
    first, count = s["q_start"][:-1].long()[:, None], (s["q_start"][1:] - s["q_start"][:-1]).long()[:, None]
    live = i < count
    qi = torch.where(live, first + i, torch.zeros_like(first + i))                   # [b, t]
    pos = torch.where(live, s["q_pos"].long()[qi], torch.zeros_like(qi))
    hidden = (j[None, None, :] > pos[:, :, None])[:, :, None, :]                     # [b, t, 1, n]
    out = torch.empty(s["nq"], hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["nq"], hq, dtype=torch.float32, device=DEV)
    for h in range(hkv):
        k, v = _gather(s, s["k"], s["k_scale"], row, h), _gather(s, s["v"], s["v_scale"], row, h)
        q = s["q"][qi, h * g:(h + 1) * g].float() * s["sm_scale"]                    # [b, t, g, d]
        p = torch.matmul(q.reshape(b, t * g, d), k.transpose(1, 2)).view(b, t, g, n)
        p.masked_fill_(hidden, -math.inf)
        m = p.amax(-1, keepdim=True)
        p.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(b, t * g, n), v).view(b, t, g, d) / total
        out[qi[live], h * g:(h + 1) * g] = o[live].bfloat16()
        lse[qi[live], h * g:(h + 1) * g] = (m + total.log())[..., 0][live]
    return {"out": out, "lse": lse}


def _touched(s):
    """(sequence, block, keys in it) of the blocks with new tokens."""
    blk = s["case"]["block"]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    ctx = s["ctx"].long()
    lo, hi = (ctx - n) // blk, (ctx - 1) // blk
    count = torch.where(n > 0, hi - lo + 1, torch.zeros_like(n))
    most = (s["max_new"] + blk - 2) // blk + 1
    i = lo[:, None] + torch.arange(most, device=DEV)
    at = torch.nonzero(torch.arange(most, device=DEV) < count[:, None])
    b, i = at[:, 0], i[at[:, 0], at[:, 1]]
    return b, i, torch.clamp(ctx[b] - i * blk, max=blk)


def _select_plain(s):
    c = s["case"]
    blk, nsel, hq, hkv, d = c["block"], c["nsel"], c["hq"], c["hkv"], c["d"]
    b, i, n = _touched(s)
    x = torch.arange(blk, device=DEV)
    j = i[:, None] * blk + torch.minimum(x, (n - 1)[:, None])       # the last key again behind the last
    row = _rows(s, b[:, None], j)
    at = row[:, 0] // blk
    for h in range(hkv):
        k = _gather(s, s["k"], s["k_scale"], row, h)                # [m, blk, d]
        lo, hi = k.amin(1), k.amax(1)
        top = torch.maximum(lo.abs(), hi.abs()).amax(-1)
        sc = torch.where(top > 0, _pow2_above(top / 127.0), torch.ones_like(top))
        s["bounds"][at, h, 0] = torch.floor(lo / sc[:, None]).to(torch.int8)
        s["bounds"][at, h, 1] = torch.ceil(hi / sc[:, None]).to(torch.int8)
        s["bound_scale"][at, h] = sc
    # padded to the longest sequence and the most new tokens, in pieces of sequences and tokens
    g, width, most = hq // hkv, (s["max_ctx"] + blk - 1) // blk, s["max_new"]
    j = torch.arange(width, device=DEV)
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    seqs = max(1, min(c["b"], (1 << 28) // (hq * min(most, 64) * width)))
    step = max(1, (1 << 28) // (hq * seqs * width))
    s["blocks"].fill_(-1)
    for b in range(0, c["b"], seqs):
        n = count[b:b + seqs, None]
        sb = torch.arange(b, b + len(n), device=DEV)[:, None]
        used = torch.where(j * blk < s["ctx"][sb], j, torch.zeros_like(j))
        block = _rows(s, sb, used * blk) // blk                                 # [b, width]
        bounds, scale = s["bounds"][block].float(), s["bound_scale"][block]
        for i in range(0, most, step):
            x = torch.arange(i, min(i + step, most), device=DEV)
            live = x < n                                                        # [b, t]
            row = torch.where(live, s["q_start"][sb].long() + x, torch.zeros_like(x))
            q = s["q"][row].float().view(len(n), -1, hkv, g, d)
            top = q.abs().amax((-1, -2), keepdim=True)
            q = torch.round(q / torch.where(top > 0, _pow2_above(top / 127.0), torch.ones_like(top)))
            z = torch.einsum("btkgd,bwkd->btkgw", q.clamp(min=0), bounds[:, :, :, 1]) \
                + torch.einsum("btkgd,bwkd->btkgw", q.clamp(max=0), bounds[:, :, :, 0])
            z = z.amax(3) * scale.transpose(1, 2)[:, None]                      # [b, t, hkv, width]
            own_block = (s["q_pos"][row].long() // blk)[..., None, None]
            sure = ((j < c["first"]) | (j > own_block - c["local"])) & (j <= own_block)
            z.masked_fill_(sure, math.inf).masked_fill_(j > own_block, -math.inf)
            order = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :nsel]
            kept = order.masked_fill(order > own_block, 1 << 30).sort(-1).values
            kept = kept.masked_fill(kept == 1 << 30, -1).int()
            s["blocks"][row[live], :, :kept.shape[-1]] = kept[live]
    pos = s["q_pos"].long()
    n = torch.clamp(pos // blk + 1, max=nsel)
    s["sel_len"].copy_(((n - 1) * blk + pos % blk + 1).int()[:, None].expand(s["nq"], hkv))
    return {n: s[n] for n in ("bounds", "bound_scale", "blocks", "sel_len")}


def _attend_plain(s):
    c = s["case"]
    blk, nsel, hq, hkv, d = c["block"], c["nsel"], c["hq"], c["hkv"], c["d"]
    g, nq, n = hq // hkv, s["nq"], c["nsel"] * blk
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(count), device=DEV), count, output_size=nq)
    out = torch.empty(nq, hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(nq, hq, dtype=torch.float32, device=DEV)
    x = torch.arange(n, device=DEV)
    step = max(1, (1 << 29) // (n * d))
    for h in range(hkv):
        for i in range(0, nq, step):
            e = min(nq, i + step)
            j = s["blocks"][i:e, h].long()[:, x // blk] * blk + x % blk
            seen = x < s["sel_len"][i:e, h, None]
            row = _rows(s, seq[i:e, None], torch.where(seen, j, torch.zeros_like(j)))
            k, v = _gather(s, s["k"], s["k_scale"], row, h), _gather(s, s["v"], s["v_scale"], row, h)
            q = s["q"][i:e, h * g:(h + 1) * g].float() * s["sm_scale"]
            p = torch.matmul(q, k.transpose(1, 2))
            p.masked_fill_(~seen[:, None], -math.inf)
            m = p.amax(-1, keepdim=True)
            p.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            out[i:e, h * g:(h + 1) * g] = (torch.matmul(p, v) / total).bfloat16()
            lse[i:e, h * g:(h + 1) * g] = (m + total.log())[..., 0]
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
def exact(c, seed):
    if work(c)["flops"] > 9e12:
        return None
    s = prepare(c, seed)
    return {"plan": _plan_exact, "insert": _insert_exact, "decode": _dense_exact, "prompt": _dense_exact,
            "select": _select_exact, "attend": _attend_exact}[c["op"]](s)


def _plan_exact(s):
    """Request by request, on the host."""
    c = s["case"]
    page = c["page"]
    table, free = s["page_table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    at = int(s["free_range"][0])
    slot, pos, start, ctx = [], [], [0], []
    for b, (p, n) in enumerate(zip(*s["lens"])):
        for col in range(-(-p // page), -(-(p + n) // page)):
            table[b, col] = free[at]
            at += 1
        j = np.arange(p, p + n)
        pos.append(j)
        slot.append(table[b, j // page].astype(np.int64) * page + j % page)
        start.append(start[-1] + n)
        ctx.append(p + n)
    rest = np.full(c["spare"], -1)
    return {"page_table": _i32(table), "ctx": _i32(ctx), "q_start": _i32(start),
            "q_pos": _i32(np.concatenate(pos + [rest])),
            "slot": torch.from_numpy(np.concatenate(slot + [rest]).astype(np.int64)).to(DEV),
            "next": _i32([at, int(s["free_range"][1])])}


def _spot(s, b, j):
    """Physical rows of tokens j (host array) of sequence b, as a tensor."""
    page = s["case"]["page"]
    j = torch.as_tensor(np.asarray(j), device=DEV)
    return s["page_table"][b].long()[torch.div(j, page, rounding_mode="floor")] * page + j.remainder(page)


def _insert_exact(s):
    c = s["case"]
    rot, sb, nq = c["rot"], c["sb"], s["nq"]

    def turned(x):
        x = x.double()
        if not rot:
            return x
        z = torch.polar(torch.ones(nq, rot // 2, dtype=torch.float64, device=DEV),
                        s["q_pos"].double().outer(s["inv_freq"].double()))
        part = x[..., :rot].reshape(nq, x.shape[1], 2, rot // 2).transpose(-1, -2) if c["half"] \
            else x[..., :rot].reshape(nq, x.shape[1], rot // 2, 2)
        w = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None])
        w = w.transpose(-1, -2) if c["half"] else w
        return torch.cat([w.reshape(nq, x.shape[1], rot), x[..., rot:]], -1)

    r = {"q": turned(s["q"])}
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        code = s[name + "_cache"].view(torch.float8_e4m3fn).double()
        scale = s[name + "_scale"].double()
        at = 0
        for b, (p, n) in enumerate(zip(*s["lens"])):
            for lo in range(p // sb * sb, p + n if n else 0, sb):
                first, last = max(lo, p), min(lo + sb, p + n)     # the block's new tokens
                y = x[at + first - p:at + last - p]
                need = (y.abs().amax((0, 2)) / E4M3_MAX).clamp(min=LEAST_SCALE)
                need = _power64(torch.ceil(torch.log2(need)))
                # (a logarithm of 64 bits may round up across a power of two)
                need = torch.where(need / 2 * E4M3_MAX >= y.abs().amax((0, 2)).clamp(min=LEAST_SCALE * E4M3_MAX),
                                   need / 2, need)
                rows = _spot(s, b, np.arange(lo, last))
                home = rows[0] // sb
                if first > lo:
                    need = torch.maximum(need, scale[home])
                    code[rows[:first - lo]] *= (scale[home] / need)[:, None]
                scale[home] = need
                code[rows[first - lo:]] = y / need[:, None]
            at += n
        r[name], r[name + "_scale"] = code, scale
    return r


def _values64(s, x, scale, rows):
    """fp64 [len(rows), hkv, d]"""
    c = s["case"]
    if c["kv"] == "bf16":
        return x[rows].double()
    at = rows if c["kv"] == "row" else torch.div(rows, c["sb"], rounding_mode="floor")
    return x[rows].view(torch.float8_e4m3fn).double() * scale[at].double()[..., None]


def _dense_exact(s):
    """Sequence by sequence, key head by key head, a block of new tokens at a time."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    out = torch.zeros(s["nq"], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["nq"], hq, dtype=torch.float64, device=DEV)
    at = 0
    for b, (p, m) in enumerate(zip(*s["lens"])):
        rows = _spot(s, b, np.arange(p + m))
        tok = torch.arange(p + m, device=DEV)
        kk, vv = _values64(s, s["k"], s["k_scale"], rows), _values64(s, s["v"], s["v_scale"], rows)
        for h in range(hkv):
            for i in range(0, m, 512):
                e = min(m, i + 512)
                seen = p + e                                      # keys that the block's last token sees
                z = torch.einsum("tgd,nd->tgn", s["q"][at + i:at + e, h * g:(h + 1) * g].double(), kk[:seen, h])
                z *= s["sm_scale"]
                late = tok[None, :seen] > torch.arange(p + i, p + e, device=DEV)[:, None]
                z[late[:, None, :].expand_as(z)] = -math.inf
                top = torch.logsumexp(z, -1)
                lse[at + i:at + e, h * g:(h + 1) * g] = top
                out[at + i:at + e, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", torch.exp(z - top[..., None]),
                                                                     vv[:seen, h])
        at += m
    return {"out": out, "lse": lse}


def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _step64(top):
    """2^e with 127 2^e >= top > 127 2^(e - 1), 1 for zeros."""
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 127.0))
    p = _power64(e)
    p = torch.where(127.0 * p / 2 >= top, p / 2, p)
    p = torch.where(127.0 * p < top, p * 2, p)
    return torch.where(top > 0, p, torch.ones_like(p))


def _select_exact(s):
    c = s["case"]
    blk, nsel, hq, hkv, d = c["block"], c["nsel"], c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    bounds, scale = s["bounds"].clone(), s["bound_scale"].clone()
    blocks = torch.full((s["nq"], hkv, nsel), -1, dtype=torch.int32, device=DEV)
    sel_len = torch.zeros(s["nq"], hkv, dtype=torch.int32, device=DEV)
    at = 0
    for b, (p, m) in enumerate(zip(*s["lens"])):
        for i in range(p // blk, (p + m - 1) // blk + 1 if m else 0):
            rows = _spot(s, b, np.arange(i * blk, min((i + 1) * blk, p + m)))
            k = _values64(s, s["k"], s["k_scale"], rows).float().double()  # a key's value is an fp32 number
            sc = _step64(k.abs().amax((0, 2)))
            home = rows[0] // blk
            bounds[home, :, 0] = torch.floor(k.amin(0) / sc[:, None]).to(torch.int8)
            bounds[home, :, 1] = torch.ceil(k.amax(0) / sc[:, None]).to(torch.int8)
            scale[home] = sc.float()
        if not m:
            continue
        width = (p + m - 1) // blk + 1
        home = torch.div(_spot(s, b, np.arange(width) * blk), blk, rounding_mode="floor")
        lo, hi, w = bounds[home, :, 0].double(), bounds[home, :, 1].double(), scale[home].double()
        q = s["q"][at:at + m].double().view(m, hkv, g, d)
        q = torch.round(q / _step64(q.abs().amax((2, 3)))[:, :, None, None])
        for i in range(0, m, 256):
            e = min(m, i + 256)
            mid, half = (lo + hi) / 2, (hi - lo) / 2               # max(q lo, q hi) = q mid + |q| half
            z = torch.einsum("tkgd,wkd->tkgw", q[i:e], mid) + torch.einsum("tkgd,wkd->tkgw", q[i:e].abs(), half)
            z = z.max(2).values * w.t()
            for h in range(hkv):
                x, j = z[:, h], torch.arange(width, device=DEV)
                pos = torch.arange(p + i, p + e, device=DEV)
                mine = pos[:, None] // blk
                key = torch.where((j < c["first"]) | (j > mine - c["local"]), torch.full_like(x, 1e30), x)
                key = torch.where(j > mine, torch.full_like(x, -1e30), key)
                # by score, then by block: a stable ascending sort of the reversed order, reversed
                turn = torch.sort(key.flip(-1), dim=-1, stable=True).indices
                best = (width - 1 - turn).flip(-1)[:, :nsel]
                best = torch.where(best > mine, torch.full_like(best, width), best).sort(-1).values
                n = best.shape[1]
                blocks[at + i:at + e, h, :n] = torch.where(best == width, torch.full_like(best, -1), best).int()
                n = torch.clamp(mine[:, 0] + 1, max=nsel)
                sel_len[at + i:at + e, h] = ((n - 1) * blk + pos % blk + 1).int()
        at += m
    return {"bounds": bounds, "bound_scale": scale.double(), "blocks": blocks, "sel_len": sel_len}


def _attend_exact(s):
    """Token by token, the selected keys of all heads at once where heads' lists differ by the head alone."""
    c = s["case"]
    blk, hq, hkv, d = c["block"], c["hq"], c["hkv"], c["d"]
    g, page = hq // hkv, c["page"]
    out = torch.zeros(s["nq"], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["nq"], hq, dtype=torch.float64, device=DEV)
    heads = torch.arange(hkv, device=DEV)[:, None]
    lists, at = s["blocks"].long(), 0
    for b, (p, m) in enumerate(zip(*s["lens"])):
        for t in range(at, at + m):
            n, seen = _selected(c, p + t - at)
            j = (lists[t, :, :n, None] * blk + torch.arange(blk, device=DEV)).view(hkv, n * blk)[:, :seen]
            rows = s["page_table"][b].long()[j // page] * page + j % page         # [hkv, seen]
            kv = []
            for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
                y = x[rows, heads]
                if c["kv"] == "bf16":
                    kv.append(y.double())
                else:
                    sc = scale[rows if c["kv"] == "row" else rows // c["sb"], heads].double()
                    kv.append(y.view(torch.float8_e4m3fn).double() * sc[..., None])
            z = torch.bmm(s["q"][t].double().view(hkv, g, d), kv[0].transpose(1, 2)) * s["sm_scale"]
            top = torch.logsumexp(z, -1)
            lse[t] = top.view(hq)
            out[t] = torch.bmm(torch.exp(z - top[..., None]), kv[1]).view(hq, d)
        at += m
    return {"out": out, "lse": lse}

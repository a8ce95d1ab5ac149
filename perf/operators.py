"""Dense grouped-query attention beside the sparse layer: what is measured.

Three operators that a layer without an indexer needs (the dense layers that
hybrid sparse models keep):

- insert  dsa_kv_insert: new tokens' keys and values into their caches, the
          keys' and queries' position rotation applied on the way;
- decode  dense_gqa_decode: one or a few new tokens per sequence over a long
          cache, split over the cache's length and joined;
- prompt  dense_gqa_prefill: whole prompts, causal, grouped heads, packed
          sequences of different lengths, with or without earlier tokens.

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


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one decode step of 64 sequences: the layer's smallest call, all latency
        dict(name="insert 64 tokens", op="insert", n=64, hq=64, hkv=8, d=128, kv="bf16", rot=64, half=False,
             fused=True),
        # a prompt chunk into an 8-bit cache, slices of one fused projection
        dict(name="insert 8191 e4m3", op="insert", n=8191, hq=64, hkv=8, d=128, kv="e4m3", rot=128, half=True,
             fused=True),
        # keys and values of many prompts at once (queries rotated elsewhere)
        dict(name="insert 131072 kv", op="insert", n=131072, hq=0, hkv=8, d=128, kv="bf16", rot=64, half=True,
             fused=False),
        # one user, a short chat: a single sequence has to fill the GPU
        dict(name="decode 1x4096", op="decode", b=1, ctx0=4096, ctx1=4096, t=1, hq=64, hkv=8, d=128, kv="bf16",
             page=64),
        # the batch and context of the sparse layer's paged benchmark
        dict(name="decode 64x32768", op="decode", b=64, ctx0=32768, ctx1=32768, t=1, hq=64, hkv=8, d=128, kv="bf16",
             page=64),
        # speculative verification, four tokens each, contexts of very different lengths, 8-bit cache
        dict(name="decode 128x4 ragged e4m3", op="decode", b=128, ctx0=61, ctx1=16381, t=4, hq=64, hkv=8, d=128,
             kv="e4m3", page=64),
        # one very long context in an 8-bit cache
        dict(name="decode 1x524288 e4m3", op="decode", b=1, ctx0=524288, ctx1=524288, t=1, hq=64, hkv=8, d=128,
             kv="e4m3", page=64),
        # many short chats, ungrouped small heads, contiguous caches
        dict(name="decode 256 short d64", op="decode", b=256, ctx0=1, ctx1=2049, t=1, hq=32, hkv=32, d=64, kv="bf16",
             page=0),
        # a few short prompts: latency
        dict(name="prompt 8 short d64", op="prompt", b=8, len0=5, len1=131, past=0, hq=32, hkv=4, d=64, kv="bf16",
             page=0, fused=True),
        # a packed batch of prompts of different lengths
        dict(name="prompt 24 packed", op="prompt", b=24, len0=17, len1=4095, past=0, hq=64, hkv=8, d=128, kv="bf16",
             page=0, fused=True),
        # one long prompt
        dict(name="prompt 1x16384", op="prompt", b=1, len0=16384, len1=16384, past=0, hq=64, hkv=8, d=128, kv="bf16",
             page=0, fused=False),
        # a chunk of a long prompt over the paged cache that holds the tokens before it
        dict(name="prompt chunk 2048 of 65536", op="prompt", b=1, len0=2048, len1=2048, past=63488, hq=64, hkv=8,
             d=128, kv="bf16", page=64, fused=False),
    ]


HEADS = [(64, 8), (32, 4), (32, 32), (16, 2), (12, 4), (40, 8), (8, 1), (5, 5), (14, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["insert", "decode", "decode", "prompt", "prompt"])
    hq, hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, 16, 64, 64, 128, 256])
    if op == "insert":
        n = _log(rng, 1, 131072)
        hq = rng.choice([0, hq])
        while n * (hq + 2 * hkv) * d > 131072 * 16 * 128:  # no dearer than the largest listed insert
            n = (n + 1) // 2
        return dict(op=op, n=n, hq=hq, hkv=hkv, d=d, kv=rng.choice(["bf16", "e4m3"]),
                    rot=rng.choice([0, 16, 32, d // 2, d, d]), half=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "decode":
        b, t = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 5])
        ctx1 = _log(rng, 8, 524288)
        while b * ctx1 * hkv * d > 64 * 32768 * 8 * 128 // 2:
            b, ctx1 = (b + 1) // 2, max(8, ctx1 * 3 // 4)
        ctx0 = rng.choice([ctx1, max(t, ctx1 // 2), t])
        return dict(op=op, b=b, ctx0=ctx0, ctx1=ctx1, t=t, hq=hq, hkv=hkv, d=d, kv=rng.choice(["bf16", "e4m3"]),
                    page=page)
    b, len1 = _log(rng, 1, 32), _log(rng, 1, 8192)
    past = rng.choice([0, 0, _log(rng, 1, 32768)])
    while b * len1 * (len1 + past) * hq * d > 2048 * 65536 * 64 * 128 // 4 or b * (len1 + past) > 131072:
        b, len1, past = (b + 1) // 2, (len1 * 3 + 3) // 4, past * 3 // 4
    return dict(op=op, b=b, len0=rng.choice([1, max(1, len1 // 2), len1]), len1=len1, past=past, hq=hq, hkv=hkv, d=d,
                kv=rng.choice(["bf16", "bf16", "e4m3"]) if past else "bf16", page=page if past else 0,
                fused=False if past else rng.random() < 0.5)


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread (the longest first)."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(c):
    """(tokens in the cache, new tokens) of each sequence, before the shuffle."""
    if c["op"] == "decode":
        ctx = _spread(c["ctx0"], c["ctx1"], c["b"])
        return ctx, [min(c["t"], x) for x in ctx]
    new = _spread(c["len0"], c["len1"], c["b"])
    return [x + c["past"] for x in new], new


def work(c):
    el = 1 if c["kv"] == "e4m3" else 2
    per_tok = 2 * c["hkv"] * (c["d"] * el + (4 if el == 1 else 0))  # a token's keys and values in the cache
    if c["op"] == "insert":
        rows = c["n"]
        moved = rows * (2 * c["hkv"] * c["d"] * 2 + per_tok + 2 * c["hq"] * c["d"] * 2 + 12)
        return {"bytes": moved, "flops": 3 * rows * c["rot"] * (c["hq"] + c["hkv"])}
    ctx, new = _lengths(c)
    nq = sum(new)
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(ctx, new))
    kv = sum(ctx) * per_tok
    return {"bytes": kv + nq * c["hq"] * (4 * c["d"] + 4), "flops": 4 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------------------
# inputs
def _normal(gen, *shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=gen)


def _codes(gen, *shape):
    """e4m3 codes of normal values with amax/448 scales: most of a row's codes are large."""
    x = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):  # a piece at a time: the fp32 values are four times the codes
        part = torch.empty(min(1 << 28, flat.numel() - i), dtype=torch.float32, device=DEV).normal_(generator=gen)
        flat[i:i + part.numel()] = (part * 150.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _tokens(gen, n, hq, hkv, d, fused):
    """q, k, v [n, heads, d] of new tokens: slices of one projection, or tensors of their own."""
    if fused:
        x = _normal(gen, n, hq + 2 * hkv, d)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (_normal(gen, n, hq, d) if hq else None), _normal(gen, n, hkv, d), _normal(gen, n, hkv, d)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 31))
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    e4m3 = c["kv"] == "e4m3"
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device=DEV))

    def i32(v):
        return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)

    if c["op"] == "insert":
        n = c["n"]
        pages = (n + 63) // 64 + 7  # 64-token pages in a random order, a few of them not written
        order = rng.permutation(pages)
        slot = (order[np.arange(n) // 64] * 64 + np.arange(n) % 64).astype(np.int64)
        rows = pages * 64
        s["q"], s["k"], s["v"] = _tokens(gen, n, hq, hkv, d, c["fused"])
        if not hq:
            s["q"] = None
        s["slot"] = torch.from_numpy(slot).to(DEV)
        s["pos"] = i32(rng.randint(0, 131072, n))
        s["inv_freq"] = None
        if c["rot"]:
            i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-i / c["rot"])).float().to(DEV)
        make = _codes if e4m3 else _normal
        s["k_cache"], s["v_cache"] = make(gen, rows, hkv, d), make(gen, rows, hkv, d)
        s["k_scale"] = s["v_scale"] = None
        if e4m3:
            s["k_scale"] = torch.rand(rows, hkv, generator=gen, device=DEV) * 0.004 + 0.004
            s["v_scale"] = torch.rand(rows, hkv, generator=gen, device=DEV) * 0.004 + 0.004
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV) if hq else None
        if own:
            import dsa_sparse_mla_query_gb300 as dsa
            s["shape"] = dsa.GqaShape(max(hq, hkv), hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16)
        return s

    ctx, new = _lengths(c)
    order = rng.permutation(c["b"])
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    q_start = np.concatenate([[0], np.cumsum(new)])
    nq = int(q_start[-1])
    s.update(nq=nq, max_ctx=max(ctx), max_new=max(new), ctx=i32(ctx), q_start=i32(q_start),
             q_pos=i32(np.concatenate([np.arange(n - m, n) for n, m in zip(ctx, new)])),
             page_table=None, seq_base=None, sm_scale=1.0 / math.sqrt(d), lens=(ctx, new))
    if c["page"]:
        used = [(x + c["page"] - 1) // c["page"] for x in ctx]
        order = rng.permutation(sum(used))
        table = np.zeros((c["b"], max(used)), np.int32)
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = order[at:at + u]
            at += u
        rows = sum(used) * c["page"]
        s["page_table"] = i32(table)
    else:
        base = np.concatenate([[0], np.cumsum(ctx)])
        rows = int(base[-1])
        s["seq_base"] = torch.from_numpy(base[:-1].astype(np.int64)).to(DEV)
    s["rows"] = rows
    s["k_scale"] = s["v_scale"] = None
    if c["op"] == "prompt" and c["fused"]:
        s["q"], s["k"], s["v"] = _tokens(gen, nq, hq, hkv, d, True)
    elif e4m3:
        s["q"] = _normal(gen, nq, hq, d)
        s["k"], s["v"] = _codes(gen, rows, hkv, d), _codes(gen, rows, hkv, d)
        s["k_scale"] = torch.rand(rows, hkv, generator=gen, device=DEV) * 0.004 + 0.004
        s["v_scale"] = torch.rand(rows, hkv, generator=gen, device=DEV) * 0.004 + 0.004
    else:
        s["q"] = _normal(gen, nq, hq, d)
        s["k"], s["v"] = _normal(gen, rows, hkv, d), _normal(gen, rows, hkv, d)
    if own:
        import dsa_sparse_mla_query_gb300 as dsa
        s["shape"] = dsa.GqaShape(hq, hkv, d, dsa.DSA_FP8_E4M3_ROWSCALE if e4m3 else dsa.DSA_BF16,
                                  q_stride=s["q"].stride(0), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        s["seqs"] = dsa.Seqs(s["ctx"], s["q_start"], s["q_pos"], max_ctx=s["max_ctx"], max_q_per_seq=s["max_new"],
                             num_rows=rows, page_table=s["page_table"], page_size=c["page"], seq_base=s["seq_base"])
        s["ws_bytes"] = dsa.dense_gqa_workspace_size(s["shape"], s["seqs"], nq)
        s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty(nq, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(nq, hq, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
def run(s):
    if own:
        return _run_own(s)
    if s["case"]["op"] == "insert":
        return _insert_plain(s)
    return _attend_plain(s)


def _run_own(s):
    import dsa_sparse_mla_query_gb300 as dsa
    c = s["case"]
    if c["op"] == "insert":
        q, k, v = s["q"], s["k"], s["v"]
        dsa.dsa_kv_insert(s["shape"], k, v, q, s["pos"], s["slot"], c["n"], s["inv_freq"], c["rot"],
                          dsa.DSA_ROPE_HALVES if c["half"] else dsa.DSA_ROPE_PAIRS, s["k_cache"], s["v_cache"],
                          s["k_scale"], s["v_scale"], s["k_cache"].shape[0], s["q_out"], k_stride=k.stride(0),
                          v_stride=v.stride(0), q_stride=0 if q is None else q.stride(0), d_status=s["status"])
        return _inserted(s)
    attend = dsa.dense_gqa_decode if c["op"] == "decode" else dsa.dense_gqa_prefill
    attend(s["shape"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["seqs"], s["nq"], s["sm_scale"],
           s["out"], s["lse"], s["ws"], s["ws_bytes"], d_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _inserted(s):
    """The caches (e4m3 codes as the values they stand for), their scales and the rotated queries."""
    if s["k_scale"] is None:
        r = {"k": s["k_cache"], "v": s["v_cache"]}
    else:
        r = {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
             "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if s["q_out"] is not None:
        r["q"] = s["q_out"]
    return r


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


def _store_plain(x, slot, cache, scale):
    if scale is None:
        cache[slot] = x.to(cache.dtype)
        return
    amax = x.abs().amax(-1)
    sc = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    scale[slot] = sc
    cache[slot] = (x / sc[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _insert_plain(s):
    c = s["case"]
    k = _rotate_plain(s["k"].float(), s["pos"], s["inv_freq"], c["rot"], c["half"])
    _store_plain(k, s["slot"], s["k_cache"], s["k_scale"])
    _store_plain(s["v"].float(), s["slot"], s["v_cache"], s["v_scale"])
    if s["q"] is not None:
        s["q_out"] = _rotate_plain(s["q"].float(), s["pos"], s["inv_freq"], c["rot"], c["half"]).bfloat16()
    return _inserted(s)


def _attend_plain(s):
    """Padded to the longest sequence and the most new tokens; one key head at a time bounds the memory."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, b, t, n = hq // hkv, c["b"], s["max_new"], s["max_ctx"]
    j = torch.arange(n, device=DEV)
    i = torch.arange(t, device=DEV)
    if s["page_table"] is not None:
        row = s["page_table"].long()[:, j // c["page"]] * c["page"] + j % c["page"]
    else:
        row = s["seq_base"][:, None] + j
    row = torch.where(j < s["ctx"][:, None], row, torch.zeros_like(row))             # [b, n]
    first, count = s["q_start"][:-1].long()[:, None], (s["q_start"][1:] - s["q_start"][:-1]).long()[:, None]
    qi = torch.where(i < count, first + i, torch.zeros_like(first + i))              # [b, t]
    pos = torch.where(i < count, s["q_pos"].long()[qi], torch.zeros_like(qi))
    hidden = (j[None, None, :] > pos[:, :, None])[:, :, None, :]                     # [b, t, 1, n]
    live = i < count
    out = torch.empty(s["nq"], hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["nq"], hq, dtype=torch.float32, device=DEV)
    for h in range(hkv):
        k, v = s["k"][row, h], s["v"][row, h]                                        # [b, n, d]
        if s["k_scale"] is not None:
            k = k.view(torch.float8_e4m3fn).float() * s["k_scale"][row, h][..., None]
            v = v.view(torch.float8_e4m3fn).float() * s["v_scale"][row, h][..., None]
        q = s["q"][qi, h * g:(h + 1) * g].float() * s["sm_scale"]                    # [b, t, g, d]
        p = torch.matmul(q.reshape(b, t * g, d), k.float().transpose(1, 2)).view(b, t, g, n)
        p.masked_fill_(hidden, -math.inf)
        m = p.amax(-1, keepdim=True)
        p.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(b, t * g, n), v.float()).view(b, t, g, d) / total
        out[qi[live], h * g:(h + 1) * g] = o[live].bfloat16()
        lse[qi[live], h * g:(h + 1) * g] = (m + total.log())[..., 0][live]
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
def exact(c, seed):
    if work(c)["flops"] > 9e12:
        return None
    s = prepare(c, seed)
    return _insert_exact(s) if c["op"] == "insert" else _attend_exact(s)


def _insert_exact(s):
    c = s["case"]
    rot, n = c["rot"], c["n"]

    def turned(x):
        x = x.double()
        if not rot:
            return x
        z = torch.polar(torch.ones(n, rot // 2, dtype=torch.float64, device=DEV),
                        s["pos"].double().outer(s["inv_freq"].double()))
        part = x[..., :rot].reshape(n, x.shape[1], 2, rot // 2).transpose(-1, -2) if c["half"] \
            else x[..., :rot].reshape(n, x.shape[1], rot // 2, 2)
        w = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None])
        w = w.transpose(-1, -2) if c["half"] else w
        return torch.cat([w.reshape(n, x.shape[1], rot), x[..., rot:]], -1)

    r = {}
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        cache = s[name + "_cache"]
        if s["k_scale"] is None:
            r[name] = cache.double().index_copy(0, s["slot"], x)
            continue
        top = x.abs().max(-1).values
        sc = torch.where(top == 0, torch.ones_like(top), top / E4M3_MAX)
        r[name] = cache.view(torch.float8_e4m3fn).double().index_copy(0, s["slot"], x / sc[..., None])
        r[name + "_scale"] = s[name + "_scale"].double().index_copy(0, s["slot"], sc)
    if s["q"] is not None:
        r["q"] = turned(s["q"])
    return r


def _attend_exact(s):
    """Sequence by sequence, key head by key head, a block of new tokens at a time."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    out = torch.zeros(s["nq"], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["nq"], hq, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(*s["lens"])):
        tok = torch.arange(n, device=DEV)
        if s["page_table"] is None:
            rows = int(s["seq_base"][b]) + tok
        else:
            rows = s["page_table"][b, tok.div(c["page"], rounding_mode="floor")].long() * c["page"] \
                + tok.remainder(c["page"])
        kk, vv = s["k"].index_select(0, rows), s["v"].index_select(0, rows)
        if s["k_scale"] is not None:
            kk, vv = kk.view(torch.float8_e4m3fn), vv.view(torch.float8_e4m3fn)
        for h in range(hkv):
            k, v = kk[:, h].double(), vv[:, h].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][rows, h, None].double(), v * s["v_scale"][rows, h, None].double()
            for i in range(0, m, 1024):
                e = min(m, i + 1024)
                seen = n - m + e                                   # keys that the block's last token sees
                z = torch.einsum("tgd,nd->tgn", s["q"][at + i:at + e, h * g:(h + 1) * g].double(), k[:seen])
                z *= s["sm_scale"]
                late = tok[None, :seen] > torch.arange(n - m + i, n - m + e, device=DEV)[:, None]
                z[late[:, None, :].expand_as(z)] = -math.inf
                top = torch.logsumexp(z, -1)
                lse[at + i:at + e, h * g:(h + 1) * g] = top
                out[at + i:at + e, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", torch.exp(z - top[..., None]),
                                                                     v[:seen])
        at += m
    return {"out": out, "lse": lse}

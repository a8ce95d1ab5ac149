"""The step's plan and the writes of block-scaled caches refuse on the host
what they cannot serve, with every reason listed (no GPU needed)."""

from __future__ import annotations

import ctypes

import pytest
import torch

from dsa_sparse_mla_query_gb300 import _binding as B
from test_gqa_abi import _attend, _insert, _seqs, lib  # noqa: F401

BLOCK = B.DSA_FP8_E4M3_BLOCKSCALE


def _shape(sb=64, **kw):
    return B.GqaShape(16, 2, 128, BLOCK, scale_block=sb, **kw)


@pytest.mark.parametrize("name", ("dense_gqa_decode", "dense_gqa_prefill"))
@pytest.mark.parametrize("sb", (0, 8, 48, 256, -64))
def test_scale_blocks(lib, name, sb):
    rc, msg = _attend(lib, name, shape=_shape(sb), ks=0x500, vs=0x600)
    assert rc == B.DSA_ERR_UNSUPPORTED and f"scale_block {sb}" in msg, msg


@pytest.mark.parametrize("name", ("dense_gqa_decode", "dense_gqa_prefill"))
def test_pages_smaller_than_a_scale_block(lib, name):
    rc, msg = _attend(lib, name, shape=_shape(64), ks=0x500, vs=0x600,
                      seqs=_seqs(page_table=0x5000, page_size=32, max_pages=4))
    assert rc == B.DSA_ERR_UNSUPPORTED and "page_size 32 below scale_block 64" in msg
    rc, msg = _attend(lib, name, shape=_shape(64))
    assert rc == B.DSA_ERR_INVALID_ARG and "k_scale is NULL" in msg and "v_scale is NULL" in msg


def test_scale_block_is_not_read_for_other_dtypes(lib):
    """The shape's earlier form ends before scale_block."""
    s, n = _seqs(), ctypes.c_size_t()
    for dtype in (B.DSA_BF16, B.DSA_FP8_E4M3_ROWSCALE):
        shape = B.GqaShape(16, 2, 128, dtype, scale_block=-5)
        assert lib.dense_gqa_workspace_size(ctypes.byref(shape), ctypes.byref(s), 2, ctypes.byref(n)) == 0


def test_the_row_scale_write_refuses_block_scales(lib):
    rc, msg = _insert(lib, shape=_shape(), ks=0x1, vs=0x1)
    assert rc == B.DSA_ERR_UNSUPPORTED and "dsa_kv_block_insert" in msg


def _block_insert(lib, shape=None, k=0x100, k_in=0, v=0x200, v_in=0, q=0x300, q_in=0, seqs=None, n=2, inv_freq=0x600,
                  rot=64, layout=0, kc=0x700, vc=0x800, ks=0x10, vs=0x20, q_out=0x900):
    shape, seqs = shape or _shape(), seqs or _seqs()
    rc = lib.dsa_kv_block_insert(ctypes.byref(shape), k, k_in, v, v_in, q, q_in, ctypes.byref(seqs), n, inv_freq, rot,
                                 layout, kc, vc, ks, vs, q_out, None, None)
    return rc, lib.dsa_last_error_string().decode()


@pytest.mark.parametrize("kw, part, status", [
    (dict(shape=B.GqaShape(16, 2, 128, B.DSA_FP8_E4M3_ROWSCALE)), "kv_dtype 1 is not DSA_FP8_E4M3_BLOCKSCALE",
     B.DSA_ERR_UNSUPPORTED),
    (dict(shape=B.GqaShape(16, 2, 128)), "kv_dtype 0 is not", B.DSA_ERR_UNSUPPORTED),
    (dict(rot=24), "rot_dims 24", B.DSA_ERR_UNSUPPORTED),
    (dict(rot=144), "rot_dims 144", B.DSA_ERR_UNSUPPORTED),
    (dict(inv_freq=None), "rot_dims 64 without inv_freq", B.DSA_ERR_INVALID_ARG),
    (dict(layout=2), "rotation layout 2", B.DSA_ERR_UNSUPPORTED),
    (dict(k_in=128), "k_in 128", B.DSA_ERR_INVALID_ARG),
    (dict(v_in=260), "v_in 260", B.DSA_ERR_INVALID_ARG),
    (dict(q_in=4), "q_in 4", B.DSA_ERR_INVALID_ARG),
    (dict(k=0x108, v=None, ks=0x2, vs=None, q_out=None), "k is not 16-byte aligned; v is NULL; k_scale is not "
     "4-byte aligned; v_scale is NULL; q_out is NULL", B.DSA_ERR_INVALID_ARG),
    (dict(q_out=0x300, q_in=4096), "q_out is q with another stride", B.DSA_ERR_INVALID_ARG),
    (dict(seqs=_seqs(page_table=0x5000, page_size=16, max_pages=4)), "page_size 16 below scale_block 64",
     B.DSA_ERR_UNSUPPORTED),
    (dict(seqs=_seqs(num_seqs=0)), "num_seqs 0", B.DSA_ERR_INVALID_ARG),
    (dict(seqs=_seqs(num_rows=1 << 31)), "num_rows", B.DSA_ERR_UNSUPPORTED),
    (dict(n=-1), "num_q -1", B.DSA_ERR_INVALID_ARG),
])
def test_block_insert_refuses(lib, kw, part, status):
    rc, msg = _block_insert(lib, **kw)
    assert rc == status and part in msg, (rc, msg)


def test_block_insert_of_nothing(lib):
    assert _block_insert(lib, n=0)[0] == 0


def _plan(lib, cached=0x100, new=0x200, n=3, free=0x300, cap=8, rng=0x400, page=64, pages=9, table=0x500, width=4,
          num_q=5, ctx=0x600, start=0x700, pos=0x800, slot=0x900, nxt=0xA00):
    rc = lib.dsa_step_plan(cached, new, n, free, cap, rng, page, pages, table, width, num_q, ctx, start, pos, slot, nxt,
                           None, None)
    return rc, lib.dsa_last_error_string().decode()


@pytest.mark.parametrize("kw, part, status", [
    (dict(n=0), "num_seqs 0", B.DSA_ERR_INVALID_ARG),
    (dict(num_q=-1), "num_q -1", B.DSA_ERR_INVALID_ARG),
    (dict(cap=-1), "free_cap -1", B.DSA_ERR_INVALID_ARG),
    (dict(page=48), "page_size 48", B.DSA_ERR_UNSUPPORTED),
    (dict(page=8), "page_size 8", B.DSA_ERR_UNSUPPORTED),
    (dict(pages=0), "num_pages 0", B.DSA_ERR_INVALID_ARG),
    (dict(width=0), "max_pages 0", B.DSA_ERR_INVALID_ARG),
    (dict(cached=None, new=0x201, slot=0x904, nxt=None), "cached_len is NULL; new_len is not 4-byte aligned; slot is "
     "not 8-byte aligned; next_range is NULL", B.DSA_ERR_INVALID_ARG),
    (dict(ctx=0x100), "an output is one of the inputs", B.DSA_ERR_INVALID_ARG),
    (dict(nxt=0x400), "an output is one of the inputs", B.DSA_ERR_INVALID_ARG),
])
def test_plan_refuses(lib, kw, part, status):
    rc, msg = _plan(lib, **kw)
    assert rc == status and part in msg, (rc, msg)


@pytest.mark.parametrize("kw, part", [
    (dict(table=0x100), "an output is one of the inputs"),          # the page table over the lengths
    (dict(table=0x2F0), "an output is one of the inputs"),          # its end in the free list
    (dict(pos=0x1F0, num_q=5), "an output is one of the inputs"),   # the positions' end in new_len
    (dict(start=0x104), "an output is one of the inputs"),
    (dict(ctx=0x608, start=0x600), "two outputs overlap"),
    (dict(pos=0x900), "two outputs overlap"),
    (dict(nxt=0x904), "two outputs overlap"),
    (dict(ctx=0x100, pos=0x900), "an output is one of the inputs; two outputs overlap"),
])
def test_plan_refuses_memory_that_overlaps(lib, kw, part):
    rc, msg = _plan(lib, **kw)
    assert rc == B.DSA_ERR_INVALID_ARG and part in msg, (rc, msg)


def test_names_are_public():
    import dsa_sparse_mla_query_gb300 as dsa
    assert dsa.DSA_FP8_E4M3_BLOCKSCALE == 4
    for name in ("dsa_step_plan", "dsa_kv_block_insert"):
        assert callable(getattr(dsa, name)) and name in dsa.__all__


def _sized(**kw):
    return dict(dict(shape=_shape(), seqs=_seqs(), n=2, block=64, nsel=4), **kw)


def _bounds(lib, shape, seqs, n, block, nsel, k=0x100, ks=0x10, bounds=0x200, steps=0x20, **kw):
    return lib.block_gqa_bounds(ctypes.byref(shape), k, ks, ctypes.byref(seqs), n, block, bounds, steps, None, None)


def _select(lib, shape, seqs, n, block, nsel, q=0x100, bounds=0x200, steps=0x20, first=1, local=1, blocks=0x300,
            length=0x400, ws=0x10000, ws_bytes=1 << 50, **kw):
    return lib.block_gqa_select(ctypes.byref(shape), q, bounds, steps, ctypes.byref(seqs), n, block, nsel, first,
                                local, blocks, length, ws, ws_bytes, None, None)


def _listed(lib, shape, seqs, n, block, nsel, q=0x100, k=0x200, v=0x300, ks=0x10, vs=0x20, blocks=0x400,
            length=0x500, scale=0.1, out=0x600, lse=None, ws=0x10000, ws_bytes=1 << 50, **kw):
    return lib.block_gqa_attend(ctypes.byref(shape), q, k, v, ks, vs, ctypes.byref(seqs), n, blocks, length, block,
                                nsel, ctypes.c_float(scale), out, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("call", (_bounds, _select, _listed))
@pytest.mark.parametrize("kw, part, status", [
    (dict(block=8), "block 8", B.DSA_ERR_UNSUPPORTED),
    (dict(block=48), "block 48", B.DSA_ERR_UNSUPPORTED),
    (dict(block=256), "block 256", B.DSA_ERR_UNSUPPORTED),
    (dict(seqs=_seqs(page_table=0x5000, page_size=64, max_pages=4), block=128), "page_size 64 below block 128",
     B.DSA_ERR_UNSUPPORTED),
    (dict(seqs=_seqs(max_ctx=1 << 24), block=16), "more than 51200 blocks", B.DSA_ERR_UNSUPPORTED),
    (dict(n=1 << 30), "exceeds 2^30 rows", B.DSA_ERR_UNSUPPORTED),
    (dict(n=-1), "num_q -1", B.DSA_ERR_INVALID_ARG),
    (dict(shape=B.GqaShape(16, 2, 96)), "head_dim 96", B.DSA_ERR_UNSUPPORTED),
    (dict(seqs=_seqs(num_seqs=0)), "num_seqs 0", B.DSA_ERR_INVALID_ARG),
])
def test_block_calls_refuse_sizes(lib, call, kw, part, status):
    rc = call(lib, **_sized(**kw))
    msg = lib.dsa_last_error_string().decode()
    assert rc == status and part in msg, (rc, msg)


@pytest.mark.parametrize("call, kw, part, status", [
    (_bounds, dict(k=0x108, ks=None, bounds=0x204, steps=None), "k_cache is not 16-byte aligned; k_scale is NULL; "
     "bounds is not 16-byte aligned; steps is NULL", B.DSA_ERR_INVALID_ARG),
    (_select, dict(q=None, bounds=0x204, blocks=0x301, length=None), "q is NULL; bounds is not 16-byte aligned; "
     "blocks is not 4-byte aligned; sel_len is NULL", B.DSA_ERR_INVALID_ARG),
    (_select, dict(nsel=0), "nsel 0", B.DSA_ERR_UNSUPPORTED),
    (_select, dict(nsel=1025), "nsel 1025", B.DSA_ERR_UNSUPPORTED),
    (_select, dict(local=0), "num_local 0", B.DSA_ERR_INVALID_ARG),
    (_select, dict(first=-1), "num_first -1", B.DSA_ERR_INVALID_ARG),
    (_select, dict(first=2, local=3), "num_first 2 and num_local 3 exceed nsel 4", B.DSA_ERR_INVALID_ARG),
    (_select, dict(ws=None), "workspace is NULL", B.DSA_ERR_WORKSPACE),
    (_select, dict(ws=0x10010), "256-byte aligned", B.DSA_ERR_WORKSPACE),
    (_select, dict(ws_bytes=100), "workspace has 100 bytes", B.DSA_ERR_WORKSPACE),
    (_listed, dict(q=0x108, k=None, vs=0x21, out=0x604, lse=0x2), "q is not 16-byte aligned; k_cache is NULL; v_scale "
     "is not 4-byte aligned; out is not 16-byte aligned; lse is not 4-byte aligned", B.DSA_ERR_INVALID_ARG),
    (_listed, dict(nsel=-1), "nsel -1", B.DSA_ERR_UNSUPPORTED),
    (_listed, dict(scale=float("inf")), "sm_scale", B.DSA_ERR_INVALID_ARG),
    (_listed, dict(ws_bytes=100), "workspace has 100 bytes", B.DSA_ERR_WORKSPACE),
])
def test_block_calls_refuse_arguments(lib, call, kw, part, status):
    rc = call(lib, **_sized(**kw))
    msg = lib.dsa_last_error_string().decode()
    assert rc == status and part in msg, (rc, msg)


def test_block_calls_of_nothing_and_their_workspace(lib):
    for call in (_bounds, _select, _listed):
        assert call(lib, **_sized(n=0)) == 0
    shape, n, last = _shape(), ctypes.c_size_t(), 0
    for num_q, ctx in ((1, 4096), (64, 4096), (64, 65536), (4096, 65536)):
        s = _seqs(max_ctx=ctx)
        assert lib.block_gqa_workspace_size(ctypes.byref(shape), ctypes.byref(s), num_q, 64, 4, ctypes.byref(n)) == 0
        assert n.value >= max(last, num_q * 2 * ctx // 64 * 4)
        last = n.value

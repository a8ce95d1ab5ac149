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


def test_names_are_public():
    import dsa_sparse_mla_query_gb300 as dsa
    assert dsa.DSA_FP8_E4M3_BLOCKSCALE == 4
    for name in ("dsa_step_plan", "dsa_kv_block_insert"):
        assert callable(getattr(dsa, name)) and name in dsa.__all__

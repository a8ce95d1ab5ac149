"""The dense attention calls refuse on the host what they cannot serve, with
every reason listed (no GPU needed), and do nothing for nothing."""

from __future__ import annotations

import ctypes

import pytest
import torch

from dsa_sparse_mla_query_gb300 import _binding as B


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("host-only checks: with a GPU a call that is not refused would launch on the made-up pointers")
    from dsa_sparse_mla_query_gb300 import build
    build.build()
    return B.load()


def _seqs(**kw):
    base = dict(num_seqs=2, max_ctx=4096, max_q_per_seq=1, page_size=0, max_pages=0, reserved=0, num_rows=8192,
                ctx_len=0x1000, q_start=0x2000, q_pos=0x3000, page_table=None, seq_base=0x4000)
    base.update(kw)
    return B.DsaSeqsC(**base)


def _attend(lib, name="dense_gqa_decode", shape=None, seqs=None, num_q=2, q=0x100, k=0x200, v=0x300, ks=None, vs=None,
            scale=0.1, out=0x400, lse=None, ws=0x10000, ws_bytes=1 << 40):
    shape = shape or B.GqaShape(16, 2, 128)
    seqs = seqs or _seqs()
    rc = getattr(lib, name)(ctypes.byref(shape), q, k, v, ks, vs, ctypes.byref(seqs), num_q, ctypes.c_float(scale),
                            out, lse, ws, ws_bytes, None, None)
    return rc, lib.dsa_last_error_string().decode()


CALLS = ("dense_gqa_decode", "dense_gqa_prefill")


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("shape, part, status", [
    (B.GqaShape(16, 2, 96), "head_dim 96", B.DSA_ERR_UNSUPPORTED),
    (B.GqaShape(16, 3, 128), "not a multiple of num_kv_heads 3", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(0, 2, 128), "num_heads 0", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(16, 0, 128), "num_kv_heads 0", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(130, 2, 128), "65 query heads", B.DSA_ERR_UNSUPPORTED),
    (B.GqaShape(16, 2, 128, B.DSA_NVFP4), "kv_dtype 3", B.DSA_ERR_UNSUPPORTED),
    (B.GqaShape(16, 2, 128, k_stride=260), "k_stride 260", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(16, 2, 128, v_stride=128), "v_stride 128", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(16, 2, 128, q_stride=-2048), "q_stride -2048", B.DSA_ERR_INVALID_ARG),
    (B.GqaShape(16, 2, 128, B.DSA_FP8_E4M3_ROWSCALE, k_stride=264), "k_stride 264", B.DSA_ERR_INVALID_ARG),
])
def test_shapes(lib, name, shape, part, status):
    rc, msg = _attend(lib, name, shape=shape, ks=0x500, vs=0x600)
    assert rc == status and part in msg, (rc, msg)
    n = ctypes.c_size_t()
    s = _seqs()
    assert lib.dense_gqa_workspace_size(ctypes.byref(shape), ctypes.byref(s), 2, ctypes.byref(n)) == status


@pytest.mark.parametrize("name", CALLS)
def test_pointers_sizes_and_workspace(lib, name):
    rc, msg = _attend(lib, name, q=None, k=0x208, v=None, out=0x404, lse=0x402,
                      seqs=_seqs(num_seqs=0, seq_base=None))
    assert rc == B.DSA_ERR_INVALID_ARG
    for part in ("q is NULL", "k_cache is not 16-byte aligned", "v_cache is NULL", "out is not 16-byte aligned",
                 "lse is not 4-byte aligned", "num_seqs 0", "seqs.seq_base"):
        assert part in msg, (part, msg)
    rc, msg = _attend(lib, name, shape=B.GqaShape(16, 2, 128, B.DSA_FP8_E4M3_ROWSCALE))
    assert rc == B.DSA_ERR_INVALID_ARG and "k_scale is NULL" in msg and "v_scale is NULL" in msg
    rc, msg = _attend(lib, name, scale=float("nan"))
    assert rc == B.DSA_ERR_INVALID_ARG and "sm_scale" in msg
    rc, msg = _attend(lib, name, seqs=_seqs(num_rows=1 << 31))
    assert rc == B.DSA_ERR_UNSUPPORTED and "num_rows" in msg
    rc, msg = _attend(lib, name, seqs=_seqs(page_table=0x5000, page_size=48, max_pages=4))
    assert rc == B.DSA_ERR_UNSUPPORTED and "page_size 48" in msg
    s, shape, n = _seqs(), B.GqaShape(16, 2, 128), ctypes.c_size_t()
    assert lib.dense_gqa_workspace_size(ctypes.byref(shape), ctypes.byref(s), 2, ctypes.byref(n)) == 0
    assert n.value > 0
    rc, msg = _attend(lib, name, ws_bytes=n.value - 1)
    assert rc == B.DSA_ERR_WORKSPACE and f"needs {n.value}" in msg
    rc, msg = _attend(lib, name, ws=0x10010)
    assert rc == B.DSA_ERR_WORKSPACE and "256-byte aligned" in msg
    rc, msg = _attend(lib, name, ws=None)
    assert rc == B.DSA_ERR_WORKSPACE and "workspace is NULL" in msg
    assert _attend(lib, name, num_q=0)[0] == 0
    assert _attend(lib, name, num_q=-1)[0] == B.DSA_ERR_INVALID_ARG


def _insert(lib, shape=None, k=0x100, k_in=0, v=0x200, v_in=0, q=0x300, q_in=0, pos=0x400, slot=0x500, n=4,
            inv_freq=0x600, rot=64, layout=0, kc=0x700, vc=0x800, ks=None, vs=None, rows=16, q_out=0x900):
    shape = shape or B.GqaShape(16, 2, 128)
    rc = lib.dsa_kv_insert(ctypes.byref(shape), k, k_in, v, v_in, q, q_in, pos, slot, n, inv_freq, rot, layout, kc, vc,
                           ks, vs, rows, q_out, None, None)
    return rc, lib.dsa_last_error_string().decode()


@pytest.mark.parametrize("kw, part, status", [
    (dict(rot=24), "rot_dims 24", B.DSA_ERR_UNSUPPORTED),
    (dict(rot=0), "rot_dims 0", B.DSA_ERR_UNSUPPORTED),
    (dict(rot=144), "rot_dims 144", B.DSA_ERR_UNSUPPORTED),
    (dict(inv_freq=None), "rot_dims 64 without inv_freq", B.DSA_ERR_INVALID_ARG),
    (dict(layout=2), "rotation layout 2", B.DSA_ERR_UNSUPPORTED),
    (dict(k_in=128), "k_in 128", B.DSA_ERR_INVALID_ARG),
    (dict(v_in=260), "v_in 260", B.DSA_ERR_INVALID_ARG),
    (dict(q_in=4), "q_in 4", B.DSA_ERR_INVALID_ARG),
    (dict(k=0x108, v=None, slot=0x504, q_out=None), "k is not 16-byte aligned; v is NULL; slot is not 8-byte aligned; "
     "q_out is NULL", B.DSA_ERR_INVALID_ARG),
    (dict(q_out=0x300, q_in=4096), "q_out is q with another stride", B.DSA_ERR_INVALID_ARG),
    (dict(shape=B.GqaShape(16, 2, 128, B.DSA_FP8_E4M3_ROWSCALE)), "k_scale is NULL", B.DSA_ERR_INVALID_ARG),
    (dict(rows=0), "num_rows 0", B.DSA_ERR_INVALID_ARG),
    (dict(n=-1), "n -1", B.DSA_ERR_INVALID_ARG),
])
def test_insert_refuses(lib, kw, part, status):
    rc, msg = _insert(lib, **kw)
    assert rc == status and part in msg, (rc, msg)


def test_insert_of_nothing(lib):
    assert _insert(lib, n=0, k=None, v=None, q=None, kc=None, vc=None)[0] == 0


def test_a_workspace_for_the_most_queries_serves_all(lib):
    """The size grows with num_q and depends on the shape, not on the sequences."""
    for shape in (B.GqaShape(64, 8, 128), B.GqaShape(5, 5, 64), B.GqaShape(64, 1, 128, B.DSA_FP8_E4M3_ROWSCALE)):
        last = 0
        for num_q in (0, 1, 4, 37, 512, 4096, 100000):
            sizes = set()
            for seqs in (_seqs(), _seqs(num_seqs=300, max_ctx=1 << 20, max_q_per_seq=64), _seqs(max_q_per_seq=5000)):
                n = ctypes.c_size_t()
                assert lib.dense_gqa_workspace_size(ctypes.byref(shape), ctypes.byref(seqs), num_q,
                                                    ctypes.byref(n)) == 0
                sizes.add(n.value)
            assert len(sizes) == 1 and max(sizes) >= last
            last = max(sizes)

"""What the paged KV-cache calls refuse, on the host, before any CUDA call."""
from __future__ import annotations

import ctypes

import pytest
import torch

import moe_decode_sigmoid_gb300 as m

A = 0x100000000   # fake device addresses: nothing is dereferenced before a launch
STEP = 0x10000000


@pytest.fixture(scope="module")
def L():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return m.lib()


def _batch(**kw):
    f = dict(n_seqs=4, max_q_len=1, page_size=16, max_pages=8, n_pages=32, q_start=A, kv_len=A + 64,
             page_table=A + 128)
    f.update(kw)
    return m._PagedBatchStruct(**f)


BAD_BATCHES = [dict(n_seqs=0), dict(n_seqs=257), dict(max_q_len=0), dict(page_size=8), dict(page_size=48),
               dict(page_size=2048), dict(max_pages=0), dict(n_pages=0), dict(max_pages=(1 << 19) + 1),
               dict(n_pages=(1 << 26) + 1), dict(q_start=None), dict(kv_len=A + 2), dict(page_table=None)]
BAD_DIMS = [(32, 4, 64), (32, 3, 128), (12, 4, 128), (64, 4, 128), (0, 0, 128), (16, 16, 128), (4, 8, 128)]


def _attend(L, fp8, dims=m.ATTN_DIMS, batch=None, T=4, q=A + STEP, k=A + 2 * STEP, v=A + 3 * STEP,
            ks=A + 4 * STEP, vs=A + 5 * STEP, sinks=None, scale=0.1, window=0, out=A + 6 * STEP,
            ws=A + 7 * STEP, wsb=None):
    b = ctypes.byref(_batch() if batch is None else batch)
    wsb = m.flint_attn_workspace_bytes() if wsb is None else wsb
    d = ctypes.byref(dims) if dims is not None else None
    if fp8:
        return L.flint_attn_paged_fp8(d, b, T, q, k, v, ks, vs, sinks, scale, window, out, ws, wsb, None)
    return L.flint_attn_paged_bf16(d, b, T, q, k, v, sinks, scale, window, out, ws, wsb, None)


def _append(L, fp8, dims=m.ATTN_DIMS, batch=None, T=4, qkv=A + STEP, qn=A + 2 * STEP, kn=A + 3 * STEP,
            theta=1e6, eps=1e-6, q=A + 4 * STEP, k=A + 5 * STEP, v=A + 6 * STEP, ks=A + 7 * STEP,
            vs=A + 8 * STEP):
    b = ctypes.byref(_batch() if batch is None else batch)
    d = ctypes.byref(dims) if dims is not None else None
    if fp8:
        return L.flint_qk_norm_rope_kv_paged_fp8(d, b, T, qkv, qn, kn, theta, eps, q, k, v, ks, vs, None)
    return L.flint_qk_norm_rope_kv_paged_bf16(d, b, T, qkv, qn, kn, theta, eps, q, k, v, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("call", [_attend, _append])
def test_dims_batch_and_rows(L, call, fp8):
    assert call(L, fp8, dims=None) == m.FLINT_ERR_INVALID_ARG
    for d in BAD_DIMS:
        assert call(L, fp8, dims=m.AttnDims(*d)) == m.FLINT_ERR_UNSUPPORTED, d
        assert m.flint_attn_workspace_bytes(m.AttnDims(*d)) == 0
    for b in BAD_BATCHES:
        assert call(L, fp8, batch=_batch(**b)) == m.FLINT_ERR_INVALID_ARG, b
    for T in (0, -1, m.PAGED_MAX_TOKENS + 1):
        assert call(L, fp8, T=T) == m.FLINT_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_arguments(L, fp8):
    bad = m.FLINT_ERR_INVALID_ARG
    for name in ("q", "k", "v", "out"):
        assert _attend(L, fp8, **{name: None}) == bad
        assert _attend(L, fp8, **{name: A + STEP * 20 + 8}) == bad
    assert _attend(L, fp8, sinks=A + 2) == bad
    assert _attend(L, fp8, window=-1) == bad
    for scale in (-0.1, float("nan"), float("inf")):
        assert _attend(L, fp8, scale=scale) == bad
    if fp8:
        assert _attend(L, fp8, ks=None) == bad
        assert _attend(L, fp8, vs=A + 4 * STEP + 2) == bad
    row = 32 * 128 * 2
    assert _attend(L, fp8, out=A + STEP) == bad                        # out on q
    assert _attend(L, fp8, out=A + STEP + 4 * row - 16) == bad         # its last bytes
    assert _attend(L, fp8, out=A + 2 * STEP + 16) == bad               # in the cache
    assert _attend(L, fp8, out=A) == bad                               # on the batch's arrays
    assert _attend(L, fp8, ws=A + 3 * STEP) == bad                     # workspace on the cache
    assert _attend(L, fp8, ws=None) == m.FLINT_ERR_WORKSPACE
    assert _attend(L, fp8, ws=A + 7 * STEP + 8) == m.FLINT_ERR_WORKSPACE
    assert _attend(L, fp8, wsb=m.flint_attn_workspace_bytes() - 1) == m.FLINT_ERR_WORKSPACE


@pytest.mark.parametrize("fp8", [False, True])
def test_append_arguments(L, fp8):
    bad = m.FLINT_ERR_INVALID_ARG
    for name in ("qkv", "qn", "kn", "q", "k", "v"):
        assert _append(L, fp8, **{name: None}) == bad
        assert _append(L, fp8, **{name: A + STEP * 20 + 8}) == bad
    for x in (-1.0, float("nan"), float("inf")):
        assert _append(L, fp8, theta=x) == bad
        assert _append(L, fp8, eps=x) == bad
    if fp8:
        assert _append(L, fp8, ks=None) == bad
        assert _append(L, fp8, vs=A + 7 * STEP + 32 * 4 * 4 - 4) == bad   # scales overlap
        assert _append(L, fp8, ks=A + 5 * STEP) == bad                    # scales in the codes
    assert _append(L, fp8, q=A + STEP + 16) == bad                        # q_out on qkv
    assert _append(L, fp8, v=A + 5 * STEP + 16) == bad                    # caches overlap
    assert _append(L, fp8, k=A + 3 * STEP) == bad                         # cache on a gain
    assert _append(L, fp8, k=A) == bad                                    # cache on the page table


def test_workspace(L):
    n = m.flint_attn_workspace_bytes()
    assert n > 0 and n == m.flint_attn_workspace_bytes(m.AttnDims(1, 1, 128))
    assert L.flint_attn_workspace_bytes(None) == 0
    assert L.flint_attn_workspace_init(None, n, None) == m.FLINT_ERR_WORKSPACE
    assert L.flint_attn_workspace_init(A, n - 1, None) == m.FLINT_ERR_WORKSPACE
    assert L.flint_attn_workspace_init(A + 8, n, None) == m.FLINT_ERR_WORKSPACE
    with pytest.raises(m.FlintError) as e:
        m.flint_attn_workspace_init(torch.zeros(n, dtype=torch.uint8))
    assert "workspace must be" in str(e.value)


def test_binding_refuses_host_tensors_and_other_batches():
    i32 = torch.int32
    with pytest.raises(m.FlintError) as e:
        m.PagedBatch(torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1, 1, dtype=i32), 16, 1)
    assert "page_table must be" in str(e.value)
    q = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    for f, n in ((m.flint_attn_paged_bf16, 2), (m.flint_attn_paged_fp8, 4)):
        with pytest.raises(m.FlintError) as e:
            f(q, *[None] * n, "batch", q, None)
        assert e.value.status == m.FLINT_ERR_INVALID_ARG and "PagedBatch" in str(e.value)
    for f, n in ((m.flint_qk_norm_rope_kv_paged_bf16, 2), (m.flint_qk_norm_rope_kv_paged_fp8, 4)):
        with pytest.raises(m.FlintError) as e:
            f(q, None, None, None, q, *[None] * n, 1e6)
        assert "PagedBatch" in str(e.value)

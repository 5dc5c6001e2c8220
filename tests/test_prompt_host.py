"""What the calls of the linear side of a prompt refuse, on the host, before any CUDA call."""
from __future__ import annotations

import ctypes

import pytest
import torch

import moe_decode_sigmoid_gb300 as m

A = 0x10000000000   # fake device addresses: nothing is dereferenced before a launch
STEP = 0x1000000000
BAD, UNSUPPORTED, WORKSPACE = (m.FLINT_ERR_INVALID_ARG, m.FLINT_ERR_UNSUPPORTED,
                               m.FLINT_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return m.lib()


def _linear(L, dims=(64, 32, 0, 0), rows=4, x=A, w=A + STEP, bias=None, res=None, out=A + 2 * STEP,
            ws=A + 3 * STEP, wsb=None):
    d = None if dims is None else ctypes.byref(m.LinearDims(*dims))
    wsb = m.flint_prompt_workspace_bytes() if wsb is None else wsb
    return L.flint_linear_bf16(d, rows, x, w, bias, res, out, ws, wsb, None)


def _grouped(L, dims=(64, 32, 0, 0), groups=4, rows=8, start=A + 4 * STEP, index=A + 5 * STEP, n_x=5,
             x=A, w=A + STEP, bias=None, out=A + 2 * STEP, ws=A + 3 * STEP, wsb=None):
    d = None if dims is None else ctypes.byref(m.LinearDims(*dims))
    wsb = m.flint_prompt_workspace_bytes() if wsb is None else wsb
    return L.flint_grouped_linear_bf16(d, groups, rows, start, index, n_x, x, w, bias, out, ws, wsb,
                                       None)


def _select(L, dims=m.FULL_DIMS, n=4, logits=A, bias=None, idx=A + STEP, w=A + 2 * STEP,
            start=A + 3 * STEP, row=A + 4 * STEP, pair=A + 5 * STEP, ws=A + 6 * STEP, wsb=None):
    wsb = m.flint_prompt_workspace_bytes() if wsb is None else wsb
    d = None if dims is None else ctypes.byref(dims)
    return L.flint_moe_select(d, n, logits, bias, idx, w, start, row, pair, ws, wsb, None)


def _combine(L, dims=m.FULL_DIMS, n=4, res=A, y=A + STEP, pair=A + 2 * STEP, w=A + 3 * STEP,
             shared=None, out=A + 4 * STEP):
    d = None if dims is None else ctypes.byref(dims)
    return L.flint_moe_combine_bf16(d, n, res, y, pair, w, shared, out, None)


def _layer(L, dims=m.FULL_DIMS, n=4, x=A, res=A + STEP, wr=A + 2 * STEP, bias=None, w13=A + 3 * STEP,
           w2=A + 4 * STEP, ws13=A + 5 * STEP, ws2=A + 6 * STEP, out=A + 7 * STEP, idx=None, w=None,
           ws=A + 8 * STEP, wsb=None):
    wsb = m.flint_prompt_workspace_bytes(4) if wsb is None else wsb
    d = None if dims is None else ctypes.byref(dims)
    return L.flint_moe_prompt_bf16(d, n, x, res, wr, bias, w13, w2, ws13, ws2, out, idx, w, ws, wsb,
                                   None)


def test_workspace_bytes(L):
    head = m.flint_prompt_workspace_bytes()
    assert 0 < head < 1 << 20
    last = head
    for n in (1, 2, 77, 8191, 8192):
        b = m.flint_prompt_workspace_bytes(n)
        assert b > last and b <= 37500 * n + (8 << 20)
        last = b
    for n in (-1, 8193, 1 << 31, 1 << 40):
        assert m.flint_prompt_workspace_bytes(n) == 0
    assert L.flint_prompt_workspace_bytes(-1) == 0 and L.flint_prompt_workspace_bytes(8193) == 0
    assert L.flint_prompt_workspace_init(None, head, None) == WORKSPACE
    assert L.flint_prompt_workspace_init(A, head - 1, None) == WORKSPACE
    assert L.flint_prompt_workspace_init(A + 8, head, None) == WORKSPACE
    assert L.flint_prompt_get_device_status(None, None) == WORKSPACE
    assert L.flint_prompt_debug_arm_stall(None, head, None) == WORKSPACE
    assert L.flint_prompt_debug_arm_stall(A, head - 1, None) == WORKSPACE


BAD_DIMS = [(0, 32, 0, 0), (60, 32, 0, 0), (m.LINEAR_MAX_IN + 8, 32, 0, 0), (64, 0, 0, 0),
            (64, 12, 0, 0), (64, m.LINEAR_MAX_OUT + 8, 0, 0), (64, 32, 4, 0), (64, 32, -1, 0),
            (64, 32, 0, 2), (64, 32, 0, -1), (64, 24, m.FLINT_ACT_SWIGLU, 0), (-8, 32, 0, 0)]


@pytest.mark.parametrize("call", [_linear, _grouped])
def test_linear_refusals(L, call):
    assert call(L, dims=None) == BAD
    for d in BAD_DIMS:
        assert call(L, dims=d) == UNSUPPORTED, d
    for rows in (0, -1, m.LINEAR_MAX_ROWS + 1):
        assert call(L, rows=rows) == BAD
    for name in ("x", "w", "out"):
        assert call(L, **{name: None}) == BAD
        assert call(L, **{name: A + 20 * STEP + 8}) == BAD
    assert call(L, bias=A + 20 * STEP + 2) == BAD
    assert call(L, ws=None) == WORKSPACE and call(L, ws=A + 20 * STEP + 8) == WORKSPACE
    assert call(L, wsb=m.flint_prompt_workspace_bytes() - 1) == WORKSPACE
    # outputs over inputs, and the workspace over anything
    for name in ("x", "w", "ws"):
        assert call(L, **{name: A + 2 * STEP + 16}) == BAD
    assert call(L, x=A + 3 * STEP + 32) == BAD
    assert call(L, bias=A + 2 * STEP) == BAD


def test_linear_residual(L):
    assert _linear(L, res=A + 20 * STEP + 8) == BAD
    # a residual that is not `out` itself may not touch it
    assert _linear(L, res=A + 2 * STEP + 16) == BAD
    assert _linear(L, res=A + 3 * STEP) == BAD


def test_grouped_refusals(L):
    for g in (0, -1, m.LINEAR_MAX_GROUPS + 1):
        assert _grouped(L, groups=g) == BAD
    for n in (0, -1, m.LINEAR_MAX_ROWS + 1):
        assert _grouped(L, n_x=n) == BAD
    assert _grouped(L, index=None, n_x=5, rows=8) == BAD
    assert _grouped(L, start=None) == BAD and _grouped(L, start=A + 2) == BAD
    assert _grouped(L, index=A + 20 * STEP + 2) == BAD
    assert _grouped(L, start=A + 2 * STEP) == BAD and _grouped(L, index=A + 2 * STEP) == BAD


@pytest.mark.parametrize("call", [_select, _combine, _layer])
def test_moe_dims_and_tokens(L, call):
    assert call(L, dims=None) == BAD
    for d in ((1024, 256, 6, 512, 1, 0), (2048, 128, 6, 512, 1, 0), (2048, 256, 8, 512, 1, 0),
              (2048, 256, 6, 256, 1, 0), (2048, 256, 6, 512, 2, 0), (2048, 256, 6, 512, 1, 2)):
        assert call(L, dims=m.Dims(*d)) == UNSUPPORTED
    for n in (0, -1, m.PAGED_MAX_TOKENS + 1):
        assert call(L, n=n) == BAD


def test_select_refusals(L):
    for name in ("logits", "idx", "w", "start", "row", "pair"):
        assert _select(L, **{name: None}) == BAD
        assert _select(L, **{name: A + 20 * STEP + 2}) == BAD
    assert _select(L, bias=A + 2) == BAD
    assert _select(L, ws=None) == WORKSPACE
    assert _select(L, wsb=m.flint_prompt_workspace_bytes() - 1) == WORKSPACE
    for a, b in (("idx", A), ("w", A + STEP), ("row", A + 5 * STEP), ("start", A + 4 * STEP),
                 ("pair", A + 6 * STEP), ("bias", A + 2 * STEP)):
        assert _select(L, **{a: b}) == BAD


def test_combine_refusals(L):
    for name in ("res", "y", "out"):
        assert _combine(L, **{name: None}) == BAD
        assert _combine(L, **{name: A + 20 * STEP + 8}) == BAD
    assert _combine(L, pair=None) == BAD and _combine(L, w=None) == BAD
    assert _combine(L, pair=A + 20 * STEP + 2) == BAD and _combine(L, shared=A + 20 * STEP + 8) == BAD
    for name in ("y", "pair", "w", "shared"):
        assert _combine(L, **{name: A + 4 * STEP}) == BAD
    assert _combine(L, res=A + 4 * STEP + 16) == BAD


def test_layer_refusals(L):
    for name in ("x", "res", "wr", "w13", "w2", "ws13", "ws2", "out"):
        assert _layer(L, **{name: None}) == BAD
        assert _layer(L, **{name: A + 20 * STEP + 8}) == BAD
    for name in ("bias", "idx", "w"):
        assert _layer(L, **{name: A + 20 * STEP + 2}) == BAD
    assert _layer(L, ws=None) == WORKSPACE
    assert _layer(L, n=5) == WORKSPACE    # of 4 tokens
    for name, at in (("x", 7), ("w13", 7), ("idx", 7), ("ws", 7), ("w2", 8), ("idx", 8), ("ws", 5)):
        assert _layer(L, **{name: A + at * STEP}) == BAD
    assert _layer(L, res=A + 7 * STEP + 16) == BAD


def test_rmsnorm_rows(L):
    d = ctypes.byref(m.FULL_DIMS)
    for n in (0, -1, m.PAGED_MAX_TOKENS + 1):
        assert L.flint_moe_rmsnorm_bf16(d, n, A, A + STEP, 1e-6, None) == BAD


def test_binding_refuses_before_the_library():
    """Tensors that are not what the header lays out: the binding names the argument."""
    x, w, out = torch.zeros(4, 64), torch.zeros(32, 64), torch.zeros(4, 32)
    ws = torch.zeros(16, dtype=torch.uint8)
    for call in (lambda: m.flint_linear_bf16(x, w, out, ws),
                 lambda: m.flint_grouped_linear_bf16(x, w[None], x, out, ws),
                 lambda: m.flint_moe_select(x, None, x, x, x, x, x, ws),
                 lambda: m.flint_moe_combine_bf16(x, x, x, x, None, x),
                 lambda: m.flint_moe_prompt_bf16(x, x, x, None, x, x, x, x, x, ws)):
        with pytest.raises(m.FlintError) as e:
            call()
        assert e.value.status == BAD
    with pytest.raises(m.FlintError):
        m.new_prompt_workspace(8193)

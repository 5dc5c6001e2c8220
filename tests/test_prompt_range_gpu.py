"""The layer of prompts over the range of its intermediates: experts' outputs of every size in
one row, of nothing but zeros, and beyond fp32's range."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p
from tests.test_moe_prompt_gpu import H, K, W_TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return fs.layer_weights(1001, fs.FULL, device="cuda")


def _run(W, x, res):
    n = len(x)
    ws, out = m.new_prompt_workspace(n), torch.empty_like(res)
    idx = torch.empty(n, K, dtype=torch.int32, device="cuda")
    wt = torch.empty(n, K, device="cuda")
    m.flint_moe_prompt_bf16(x, res, W["wr"], None, W["w13"], W["w2"], W["ws13"], W["ws2"], out, ws, idx, wt)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    return out, idx.long(), wt.double()


def _want(W, x, res, idx, wt):
    """(outputs in 64 bits, how far each may be off) for the call's own experts and weights.

    An h is off by what p.linear() says of an fp32 output, by 2^-16 of itself as a pair and as
    much for the faster silu; a y by that times |w2|, by 1040 fp32 additions (512 of hi and of
    lo), by its half step in f16, 2^-12, and by 2^-39 of the largest of its 32, whose scale it
    has; the sum by 8 fp32 additions and the output's half step."""
    def ffn(v, w13, w2):
        h, eh = p.linear(v, w13, None, None, p.SWIGLU, torch.float32)
        eh = eh + 2.0 ** -15 * (h.abs() + eh)
        w2 = w2.double().T
        y, size = h @ w2, h.abs() @ w2.abs()
        e = eh @ w2.abs() + 1040 * p.ADD * (size + eh @ w2.abs())
        big = (y.abs() + e).view(len(y), -1, 32).amax(-1).repeat_interleave(32, 1)
        return y, e + 2.0 ** -12 * (y.abs() + e) + 2.0 ** -39 * big

    y, err = ffn(x, W["ws13"][0], W["ws2"][0])
    out, size = res.double() + y, res.double().abs() + y.abs()
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        y, ey = ffn(x[t], W["w13"][e], W["w2"][e])
        out.index_add_(0, t, wt[t, j, None] * y)
        err.index_add_(0, t, wt[t, j, None] * ey)
        size.index_add_(0, t, (wt[t, j, None] * y).abs())
    err = err + 8 * 2.0 ** -24 * size
    return out, err + 2.0 ** -8 * (out.abs() + err) + 2.0 ** -126


@pytest.mark.parametrize("n", [150, 700, 4200])
def test_outputs_of_every_size(layer, n):
    """Columns of 2^-30 to 2^30 side by side, no residual: each keeps its own accuracy down to
    2^-39 of the largest of its 32."""
    x, res = fs.tokens(5000 + n, n, device="cuda")
    res.zero_()
    W = dict(layer)
    gain = 2.0 ** torch.randint(-30, 31, (H,), generator=p.gen(n), device="cuda").float()
    for k in ("w2", "ws2"):
        W[k] = (W[k] * gain[:, None].bfloat16())
    out, idx, wt = _run(W, x, res)
    p.check(out, _want(W, x, res, idx, wt))


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 60])
def test_outputs_all_small_or_large(layer, scale):
    n = 300
    x, res = fs.tokens(5001, n, device="cuda")
    res.zero_()
    W = dict(layer)
    for k in ("w2", "ws2"):
        W[k] = W[k] * scale
    out, idx, wt = _run(W, x, res)
    p.check(out, _want(W, x, res, idx, wt))


def test_outputs_of_zero(layer):
    """Columns that no expert adds to are the residual's, and do not count in their neighbours'
    scale."""
    n = 200
    x, res = fs.tokens(5002, n, device="cuda")
    W = dict(layer)
    for k in ("w2", "ws2"):
        W[k] = W[k].clone()
        W[k][:, 64:128] = 0
        W[k][:, 7] = 0
    out, idx, wt = _run(W, x, res)
    assert torch.equal(out[:, 64:128], res[:, 64:128]) and torch.equal(out[:, 7], res[:, 7])
    p.check(out, _want(W, x, res, idx, wt))


@pytest.mark.parametrize("n", [150, 4200])
def test_outputs_beyond_the_range(layer, n):
    """A column of infinities or NaN leaves the others' bits alone."""
    x, res = fs.tokens(5003 + n, n, device="cuda")
    W = dict(layer)
    bad = [5, 40, 1500]
    for k in ("w2", "ws2"):
        W[k] = W[k].clone()
        W[k][:, bad] = 0
    want, _, _ = _run(W, x, res)
    W["w2"][:, 5], W["w2"][:, 40], W["ws2"][:, 1500] = 3e38, float("nan"), float("inf")
    out, _, _ = _run(W, x, res)
    others = torch.ones(H, dtype=torch.bool, device="cuda")
    others[bad] = False
    assert torch.equal(out[:, others], want[:, others])
    assert not torch.isfinite(out[:, 5]).all() and torch.isnan(out[:, 40]).all()
    assert not torch.isfinite(out[:, 1500]).any()


@pytest.mark.parametrize("n", [129, 1001, 4096, 4097, 8192])
def test_workspace_is_enough(layer, n):
    """A call writes nothing behind the bytes that its workspace has to have, and calls of other
    sizes in the same one do not disturb it."""
    x, res = fs.tokens(5100 + n, n, device="cuda")
    size = m.flint_prompt_workspace_bytes(n)
    memory = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws, out, again = memory[:size], torch.empty_like(res), torch.empty_like(res)
    m.flint_prompt_workspace_init(ws)
    args = (layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"], layer["ws2"])
    m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    for k in (n // 2, 128, 1):
        if k > 0:
            m.flint_moe_prompt_bf16(x[:k], res[:k], *args, again[:k], ws)
    again = res.clone()
    m.flint_moe_prompt_bf16(x, again, *args, again, ws)   # in place
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    assert (memory[size:] == 0x5A).all()
    assert torch.equal(out, again)

"""Calls of the linear side of a prompt right behind the library's kernels that write what they
read, which begin before those have ended: the same bits as with a wait between the calls."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p

pytestmark = pytest.mark.gpu
BF, H, E, K = torch.bfloat16, 2048, 256, 6
TURNS = 60


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


def _empty(*s, dtype=BF):
    return torch.zeros(s, dtype=dtype, device="cuda")


def _same(turn, outs):
    """turn(i, wait, out) for other data each turn: all turns in a row, then each alone."""
    many = [[o.clone() for o in outs] for _ in range(TURNS)]
    alone = [[o.clone() for o in outs] for _ in range(TURNS)]
    torch.cuda.synchronize()
    for i in range(TURNS):
        turn(i, lambda: None, many[i])
    torch.cuda.synchronize()
    for i in range(TURNS):
        turn(i, torch.cuda.synchronize, alone[i])
    torch.cuda.synchronize()
    for i in range(TURNS):
        for a, b in zip(many[i], alone[i]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("rows", [1, 5, 8, 12, 16, 40, 300])
def test_norm_then_product(ws, rows):
    g = p.gen(rows)
    data, x = [p.bf(g, rows, H) for _ in range(TURNS)], _empty(rows, H)
    w = p.bf(g, 1040, H, scale=H ** -0.5)

    def turn(i, wait, out):
        m.flint_moe_rmsnorm_bf16(data[i], x)
        wait()
        m.flint_linear_bf16(x, w, out[0], ws)
        wait()

    _same(turn, [_empty(rows, 1040)])


@pytest.mark.parametrize("rows", [2, 16, 40])
def test_products_that_make_weights_and_bias(ws, rows):
    """A product whose weights, bias and residual are the products' right before it."""
    g = p.gen(100 + rows)
    data = [p.bf(g, 16, 64) for _ in range(TURNS)]
    u = p.bf(g, H, 64)
    x = p.bf(g, rows, H)
    xs, w, b, r = x[:, :64].contiguous(), _empty(16, H), _empty(1, 16, dtype=torch.float32), _empty(rows, 16)

    def turn(i, wait, out):
        m.flint_linear_bf16(data[i], u, w, ws)                   # w [16, H]
        wait()
        m.flint_linear_bf16(data[i][:1], data[i], b, ws)         # bias
        wait()
        m.flint_linear_bf16(xs, data[i], r, ws)                  # residual
        wait()
        m.flint_linear_bf16(x, w, out[0], ws, bias=b[0], residual=r)
        wait()

    _same(turn, [_empty(rows, 16)])


@pytest.mark.parametrize("n", [1, 9, 64, 65, 300])
def test_routing_of_a_prompt(ws, n):
    """Scores, selection, products by expert over its groups and rows, combine."""
    g = p.gen(200 + n)
    data = [p.bf(g, n, H) for _ in range(TURNS)]
    wr, w13, w2 = p.bf(g, E, H, scale=0.02), p.bf(g, E, 64, H, scale=0.02), p.bf(g, E, H, 32, scale=0.2)
    i32 = lambda *s: _empty(*s, dtype=torch.int32)  # noqa: E731
    x, logits = _empty(n, H), _empty(n, E, dtype=torch.float32)
    idx, wt = i32(n, K), _empty(n, K, dtype=torch.float32)
    start, row, pair = i32(E + 1), i32(n * K), i32(n, K)
    h, y = _empty(n * K, 32), _empty(n * K, H)

    def turn(i, wait, out):
        m.flint_moe_rmsnorm_bf16(data[i], x)
        wait()
        m.flint_linear_bf16(x, wr, logits, ws)
        wait()
        m.flint_moe_select(logits, None, idx, wt, start, row, pair, ws)
        wait()
        m.flint_grouped_linear_bf16(x, w13, start, h, ws, row_index=row, act=p.SWIGLU)
        wait()
        m.flint_grouped_linear_bf16(h, w2, start, y, ws)
        wait()
        m.flint_moe_combine_bf16(data[i], y, pair, wt, None, out[0])
        wait()

    _same(turn, [_empty(n, H)])

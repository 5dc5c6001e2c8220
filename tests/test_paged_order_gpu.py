"""GPU parity of the prompt attention where a CTA goes through many short items
in a row, pairs of tiles and split ones in turn: what orders one item's queries
behind the last one's.  Tolerances: tests/_paged.py."""
from __future__ import annotations

import pytest
import torch

from tests._paged import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    import moe_decode_sigmoid_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def ws(m):
    return m.new_attn_workspace()


def _prompts(kind, seed):
    """(new, total, window): at 8 query heads a KV head 32 tokens are a pair of
    tiles, up to 16 behind them a split item; 128 keys are a key tile."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g).tolist()  # noqa: E731
    if kind == "no context":          # one key tile: a pair, then a split item
        new = draw(33, 48, 160)
        return new, new, 0
    if kind == "two tiles, one":      # pairs of two key tiles, of one, split ones
        new = [32, 40] * 100
        return new, [200, 40] * 100, 0
    if kind == "window":              # one or two key tiles of a long context
        new = draw(20, 60, 150)
        return new, [n + c for n, c in zip(new, draw(0, 2000, 150))], 100
    new = draw(1, 70, 200)            # next tokens, drafts and prompts
    return new, [n + c for n, c in zip(new, draw(0, 300, 200))], 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv", [(32, 4), (8, 1), (16, 8)])
@pytest.mark.parametrize("kind", ["no context", "two tiles, one", "window", "mixed"])
def test_short_items_in_turn(m, ws, fmt, nq, nkv, kind):
    new, total, window = _prompts(kind, 7 + nq)
    c = Case(600 + nq, fmt, new, total, page=32, nq=nq, nkv=nkv)
    first = c.attend(m, ws, window, c.sinks)
    c.check(first, window, c.sinks)
    for _ in range(20):
        assert torch.equal(c.attend(m, ws, window, c.sinks).view(torch.int16), first.view(torch.int16))
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("total", [128, 256, 384])
def test_drafts_over_one_to_three_key_tiles(m, ws, fmt, total):
    """Split items throughout, with and without key tiles for the second half."""
    c = Case(610, fmt, [9] * 256, [total - (i % 90) for i in range(256)], page=64)
    first = c.attend(m, ws)
    c.check(first)
    for _ in range(20):
        assert torch.equal(c.attend(m, ws).view(torch.int16), first.view(torch.int16))
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK

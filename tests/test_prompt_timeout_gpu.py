"""A wait of the linear products' tiled kernel that runs out (armed by the test hook): the call
ends, its status says so, and after a new start the workspace serves again."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p

pytestmark = pytest.mark.gpu


def _plain(rows, n_out):
    g = p.gen(1)
    x, w = p.bf(g, rows, 2048), p.bf(g, n_out, 2048, scale=2048 ** -0.5)
    out = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    return (lambda ws: m.flint_linear_bf16(x, w, out, ws)), out, p.linear(x, w, None, None, p.NONE, torch.bfloat16)


def _grouped():
    g = p.gen(2)
    x, w = p.bf(g, 700, 512), p.bf(g, 2, 256, 512, scale=512 ** -0.5)
    start = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    out = torch.zeros(700, 256, dtype=torch.bfloat16, device="cuda")
    want = [p.linear(x[a:b], w[i], None, None, p.NONE, torch.bfloat16) for i, (a, b) in enumerate([(0, 300), (300, 700)])]
    return (lambda ws: m.flint_grouped_linear_bf16(x, w, start, out, ws)), out, tuple(torch.cat(t) for t in zip(*want))


# One tile a cluster with k split; one CTA a tile; pairs of CTAs; groups.
@pytest.mark.parametrize("make", [lambda: _plain(40, 512), lambda: _plain(200, 5120), lambda: _plain(4096, 4096),
                                  _grouped])
def test_a_wait_that_runs_out(make):
    from moe_decode_sigmoid_gb300 import build
    build.build()
    call, out, want = make()
    ws = m.new_prompt_workspace()
    call(ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    m.flint_prompt_debug_arm_stall(ws)
    call(ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_ERR_DEVICE_TIMEOUT
    m.flint_prompt_workspace_init(ws)
    out.zero_()
    call(ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    p.check(out, want)

"""A wait of the prompt layer's tiled kernels that runs out (armed by the test hook): the call's
other kernels end too, its status says so, and after a new start the workspace serves again."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m

pytestmark = pytest.mark.gpu


def test_a_wait_that_runs_out_in_the_layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    W, n = fs.layer_weights(1001, fs.FULL, device="cuda"), 200
    x, res = fs.tokens(1, n, device="cuda")
    ws, want, out = m.new_prompt_workspace(n), torch.empty_like(res), torch.empty_like(res)
    args = (W["wr"], None, W["w13"], W["w2"], W["ws13"], W["ws2"])
    m.flint_moe_prompt_bf16(x, res, *args, want, ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    m.flint_prompt_debug_arm_stall(ws)
    m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_ERR_DEVICE_TIMEOUT
    m.flint_prompt_workspace_init(ws)
    m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    assert torch.equal(out, want)

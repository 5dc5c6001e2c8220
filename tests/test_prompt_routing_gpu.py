"""One rule of routing for every call: a token whose experts are all masked, in the decode
call, the router, and the layer of prompts on both sides of its change of method."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p
from tests.test_moe_prompt_gpu import K, H, _layer_ref

pytestmark = pytest.mark.gpu
LOW = {"inf": float("-inf"), "lowest": torch.finfo(torch.float32).min}


@pytest.fixture(scope="module")
def layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return fs.layer_weights(1001, fs.FULL, device="cuda")


def _outputs(n):
    return (torch.full((n, H), 9.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((n, K), -9, dtype=torch.int32, device="cuda"),
            torch.full((n, K), -9.0, device="cuda"))


def _shared_only(x, res, W):
    """(residual + shared expert, how far a call may be off) in 64 bits."""
    h, eh = p.linear(x, W["ws13"][0], None, None, p.SWIGLU, torch.bfloat16)
    w2 = W["ws2"][0].double().T
    y = h @ w2
    err = eh @ w2.abs() + 528 * p.ADD * ((h.abs() + eh) @ w2.abs())
    err = err + 2.0 ** -8 * (y.abs() + err)
    out = res.double() + y
    err = err + 2.0 ** -22 * (res.double().abs() + y.abs())
    return out, err + 2.0 ** -8 * (out.abs() + err)


@pytest.mark.parametrize("low", ["inf", "lowest"])
@pytest.mark.parametrize("n", [1, 3, 8, 9, 40, 128, 129, 300])
def test_all_experts_masked(layer, n, low):
    """Weights of zeros, and an output that is the residual and the shared expert."""
    x, res = fs.tokens(4000 + n, n, device="cuda")
    offset = torch.full((256,), LOW[low], device="cuda")
    out, idx, w = _outputs(n)
    ws = m.new_prompt_workspace(n)
    m.flint_moe_prompt_bf16(x, res, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, ws, idx, w)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    assert (w == 0).all()
    assert torch.equal(idx.long(), torch.arange(K, device="cuda").expand(n, K))
    p.check(out, _shared_only(x, res, layer))


@pytest.mark.parametrize("n", [1, 5, 8, 9, 77, 256])
def test_all_experts_masked_in_decode(layer, n):
    x, res = fs.tokens(4100 + n, n, device="cuda")
    offset = torch.full((256,), float("-inf"), device="cuda")
    out, idx, w = _outputs(n)
    ws = m.new_workspace(n)
    m.flint_moe_decode_bf16(x, res, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, ws, idx, w)
    assert m.flint_moe_get_device_status(ws) == m.FLINT_OK
    assert (w == 0).all()
    p.check(out, _shared_only(x, res, layer))
    w.fill_(-9)
    m.flint_moe_route(x, layer["wr"], offset, idx, w, ws)
    assert (w == 0).all()


@pytest.mark.parametrize("n", [4, 60, 128, 129, 200])
def test_some_experts_masked(layer, n):
    """Two experts left: their weights, and zeros for the four that fill the token's choice."""
    x, res = fs.tokens(4200 + n, n, device="cuda")
    offset = torch.full((256,), LOW["lowest"], device="cuda")
    offset[[17, 250]] = torch.tensor([0.0, 50.0], device="cuda")
    out, idx, w = _outputs(n)
    m.flint_moe_prompt_bf16(x, res, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, m.new_prompt_workspace(n), idx, w)
    assert (idx[:, 0] == 250).all() and (idx[:, 1] == 17).all() and (w[:, 2:] == 0).all()
    assert torch.equal(idx[:, 2:].long(), torch.arange(4, device="cuda").expand(n, 4))
    want, err, *_ = _layer_ref(x, res, layer, offset, False)
    p.check(out, (want, err))

"""The linear calls' activations where their exponentials leave the range of fp32."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


@pytest.mark.parametrize("rows", [4, 40, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", [p.SILU, p.SWIGLU])
def test_silu_of_very_negative(ws, rows, dtype, act):
    """Gates of -60 to -103, one term a sum, so that the sums are exact; ups of 1e30, which
    bring the product back into range.

    silu(v) = v e / (1 + e), e = exp(v): e of relative error (|v| + 8) 2^-23 at most (the
    argument's rounding times |v|, and the exponential's own) and of 2^-149 where it is
    subnormal, a product, a sum and a quotient of 4 half steps, held in fp32 with steps of
    2^-149; then the product by up, and the output's half step."""
    n_out = 48
    v = torch.linspace(-60, -103, n_out, device="cuda").bfloat16()
    up = torch.full((n_out,), 1e30, device="cuda").bfloat16()
    x, w = torch.zeros(rows, 64, device="cuda").bfloat16(), torch.zeros(n_out, 64, device="cuda").bfloat16()
    x[:, 9] = 1
    w[:, 9] = v
    if act == p.SWIGLU:
        w = torch.cat([w, w.clone()])
        w[n_out:, 9] = up
    out = torch.empty(rows, n_out, dtype=dtype, device="cuda")
    m.flint_linear_bf16(x, w, out, ws, act=act)
    v, up = v.double(), up.double() if act == p.SWIGLU else torch.ones_like(up).double()
    s = v * torch.exp(v) / (1 + torch.exp(v))
    err = ((v.abs() + 8) * 2.0 ** -23 + 2.0 ** -22) * s.abs() + (v.abs() + 2) * 2.0 ** -149
    want, err = s * up, err * up
    err = err + torch.finfo(dtype).eps / 2 * (want.abs() + err) + 2.0 ** -126 * 2.0 ** -7
    p.check(out, (want.expand(rows, -1), err.expand(rows, -1)))

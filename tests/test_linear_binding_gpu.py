"""What the binding of the linear calls takes, whatever calls came before."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


@pytest.mark.parametrize("act,like", [(1.0, 1), (True, 1), (3.0, 3), (False, 0)])
def test_an_act_is_a_whole_number(ws, act, like):
    """What only equals an activation is refused, also after calls that used that one."""
    x, w = (torch.zeros(s, device="cuda").bfloat16() for s in ((4, 64), (64 if like == 3 else 32, 64)))
    out = torch.zeros(4, 32, device="cuda").bfloat16()
    start = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    m.flint_linear_bf16(x, w, out, ws, act=like)
    m.flint_grouped_linear_bf16(x, w[None], start, out, ws, act=like)
    for call in (lambda: m.flint_linear_bf16(x, w, out, ws, act=act),
                 lambda: m.flint_grouped_linear_bf16(x, w[None], start, out, ws, act=act)):
        with pytest.raises(m.FlintError) as e:
            call()
        assert e.value.status == m.FLINT_ERR_UNSUPPORTED

"""A wait of the prompt attention that runs out: the call ends, says so, writes
nothing outside its outputs, and the workspace serves again once initialised.
(The hook's barrier is one that nothing completes; every wait in the kernel ends
after a second, and so does this one.)"""
from __future__ import annotations

import time

import pytest
import torch

from tests._paged import Case, D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    import moe_decode_sigmoid_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total", [([40], [40]), ([9] * 4, [300] * 4), ([70, 300], [600, 3000]),
                                       ([20] * 200, [90] * 200)])
def test_a_wait_that_runs_out(m, fmt, new, total):
    ws = m.new_attn_workspace()
    c = Case(1000 + len(new), fmt, new, total)
    guard = torch.full((c.T + 64, c.nq, D), 7.25, dtype=torch.bfloat16, device="cuda")
    out = guard[32:32 + c.T]
    m.flint_attn_debug_arm_stall(ws)
    one = Case(1001, fmt, [1] * 3, [300, 20, 5])     # next tokens have no such wait
    one.check(one.attend(m, ws))
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK
    start = time.perf_counter()
    c.attend(m, ws, out=out)
    assert m.flint_attn_get_device_status(ws) == m.FLINT_ERR_DEVICE_TIMEOUT
    assert 0.9 < time.perf_counter() - start < 30.0
    assert (guard[:32] == 7.25).all() and (guard[32 + c.T:] == 7.25).all()
    m.flint_attn_workspace_init(ws)
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK
    out.fill_(7.25)
    c.check(c.attend(m, ws, out=out))                 # one shot
    assert torch.equal(c.attend(m, ws).view(torch.int16), out.view(torch.int16))
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK

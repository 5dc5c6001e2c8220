"""GPU parity of the paged attention at the ends of what its arguments may be."""
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


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total", [([1, 1, 1], [300, 5000, 0]), ([2, 2, 1], [300, 5000, 0]),
                                       ([20, 60, 2], [300, 5000, 1])])
def test_sinks_of_every_kind(m, ws, fmt, new, total):
    """e^sink in the denominator: none for -infinity, outputs of zero for infinity and
    for what rounds to it, NaN for NaN; a row that sees no token gets zeros whatever
    the sink."""
    c = Case(1100 + new[0], fmt, new, total)
    sinks = c.sinks.clone()
    sinks[1::8], sinks[2::8], sinks[3::8], sinks[4::8] = (float("inf"), float("-inf"), float("nan"), 3e38)
    got = c.attend(m, ws, 0, sinks)
    plain, none = c.sinks.clone(), torch.full_like(c.sinks, float("-inf"))
    ref, tol = c.reference(0, plain)
    ref_none, tol_none = c.reference(0, none)
    blind = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for s in range(c.n):
        blind[c.start[s]:c.start[s] + max(0, new[s] - total[s])] = True
    assert blind.any()
    heads = torch.arange(c.nq, device="cuda") % 8
    assert (got[blind] == 0).all()
    for kind in (1, 4):
        assert (got[:, heads == kind] == 0).all()
    assert got[~blind][:, heads == 3].isnan().all()
    off = (got.double() - ref_none).abs() - tol_none
    assert float(off[:, heads == 2].max()) <= 0.0
    off = (got.double() - ref).abs() - tol
    assert float(off[:, (heads == 0) | (heads >= 5)].max()) <= 0.0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 20])
def test_the_longest_sequence(m, ws, fmt, new):
    """2^23 tokens, the most that a row of the page table has room for."""
    c = Case(1110 + new, fmt, [new], [1 << 23], page=1024, nq=2, nkv=1, extra=1)
    c.check(c.attend(m, ws, 0, c.sinks), 0, c.sinks)
    c.check(c.attend(m, ws, 5000), 5000)
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK

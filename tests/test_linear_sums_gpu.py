"""Sums over long rows of the linear calls, where a bound on roundings is too wide to see a
missing part of k: whole numbers, whose sums are exact in fp32, have to come out exactly; and
fp32 outputs of positive terms, whose truncations in the tensor core all count the same way."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.float32)


def _rounded(want, dtype):
    """Whole numbers below 2^53, rounded once (float64 -> bf16 goes by way of fp32, which holds
    those below 2^24; products of two of them are rounded to fp32 and stop there)."""
    assert dtype is F32 or not want.numel() or float(want.abs().max()) < 2 ** 24
    return want.to(F32).to(dtype)


# Terms of at most 4: sums of 65536 stay below 2^18, and every partial sum is exact.
@pytest.mark.parametrize("n_in", [520, 1032, 2048, 4104, 8200, 32784, 65536])
@pytest.mark.parametrize("rows", [1, 16, 17, 40, 150, 700])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_whole_numbers(ws, rows, n_in, dtype):
    g = p.gen(rows + n_in)
    for n_out, bias, residual in ((264, False, False), (40, True, True)):
        x, w = _ints(g, -2, 2, rows, n_in).to(BF), _ints(g, -2, 2, n_out, n_in).to(BF)
        b = _ints(g, -1000, 1000, n_out) if bias else None
        r = _ints(g, -100, 100, rows, n_out).to(dtype) if residual else None
        out = torch.full((rows, n_out), 7.0, dtype=dtype, device="cuda")
        m.flint_linear_bf16(x, w, out, ws, bias=b, residual=r)
        want = x.double() @ w.double().T
        want = want + (b.double() if bias else 0)
        want = want + (r.double() if residual else 0)
        assert torch.equal(out, _rounded(want, dtype)), (n_out, float((out.double() - want).abs().max()))


# Gates of 2^19 and more, where silu(v) is v to the last bit: out = gate * up, rounded once.
@pytest.mark.parametrize("n_in", [520, 2048, 8200, 32784])
@pytest.mark.parametrize("rows", [3, 40, 150, 700])
def test_whole_numbers_swiglu(ws, rows, n_in):
    g = p.gen(rows + n_in + 1)
    n_out = 80
    x, w = _ints(g, -2, 2, rows, n_in).to(BF), _ints(g, -2, 2, 2 * n_out, n_in).to(BF)
    b = torch.cat([torch.full((n_out,), 2.0 ** 20, device="cuda"), torch.zeros(n_out, device="cuda")])
    out = torch.full((rows, n_out), 7.0, dtype=F32, device="cuda")
    m.flint_linear_bf16(x, w, out, ws, bias=b, act=p.SWIGLU)
    y = x.double() @ w.double().T + b.double()
    assert float(y[:, :n_out].min()) > 2 ** 19
    assert torch.equal(out, (y[:, :n_out] * y[:, n_out:]).to(F32))


@pytest.mark.parametrize("n_in", [520, 2048, 8200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[5], [0, 9, 300, 0, 33], [3, 4], [17] * 12])
def test_whole_numbers_grouped(ws, n_in, dtype, sizes):
    g = p.gen(n_in + len(sizes))
    groups, rows, n_out = len(sizes), sum(sizes), 136
    start = [sum(sizes[:i]) for i in range(groups + 1)]
    x, w = _ints(g, -2, 2, 50, n_in).to(BF), _ints(g, -2, 2, groups, n_out, n_in).to(BF)
    index = torch.randint(0, 50, (rows,), generator=g, device="cuda").to(torch.int32)
    out = torch.full((rows, n_out), 7.0, dtype=dtype, device="cuda")
    m.flint_grouped_linear_bf16(x, w, torch.tensor(start, dtype=torch.int32, device="cuda"), out, ws,
                                row_index=index)
    for i in range(groups):
        a, b = start[i], start[i + 1]
        want = x[index[a:b].long()].double() @ w[i].double().T
        assert torch.equal(out[a:b], _rounded(want, dtype)), i


@pytest.mark.parametrize("rows,n_out", [(40, 256), (150, 272), (700, 528), (4096, 256)])
@pytest.mark.parametrize("act", [p.NONE, p.SWIGLU])
def test_fp32_sums_of_positive_terms(ws, rows, n_out, act):
    """Terms that are all positive: every truncation of a partial sum counts the same way.

    An fp32 output sums at most 512 terms in the tensor core, in 32 steps of 16, each of which
    cuts at most a unit of the last place, 2^-23 of the part's sum; the 64 parts are then added
    by rounding, each addition half a unit of a sum that grows to the whole, 16 units in all, and
    twice that with k in parts over a cluster: 64 units.  One sum over all of k is off by 70
    with k in eight parts, by 210 to 560 without (measured); this one by less than 5.  SwiGLU
    doubles the bound (gate and up) and adds 16 half steps of its own."""
    n_in = 32768
    g = p.gen(rows + n_out)
    mr = n_out * (2 if act == p.SWIGLU else 1)
    x = (torch.rand(rows, n_in, generator=g, device="cuda") + 0.5).to(BF)
    w = ((torch.rand(mr, n_in, generator=g, device="cuda") + 0.5) / 256).to(BF)
    out = torch.empty(rows, n_out, dtype=F32, device="cuda")
    m.flint_linear_bf16(x, w, out, ws, act=act)
    y = x.double() @ w.double().T
    if act == p.SWIGLU:
        y = y[:, :n_out] * torch.sigmoid(y[:, :n_out]) * y[:, n_out:]
    rel = (out.double() - y).abs() / y
    units = 64 if act == p.NONE else 2 * 64 + 8
    assert float(rel.max()) <= units * 2.0 ** -23, float(rel.max()) * 2 ** 23

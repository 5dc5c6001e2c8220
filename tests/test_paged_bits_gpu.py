"""How many bits of a weight reach V in the paged attention: inputs whose outputs
are what the lower bits leave."""
from __future__ import annotations

import math

import pytest
import torch

from tests._paged import BLOCK, Case, D


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


def _held(c):
    """[rows] cache rows and positions of every sequence's tokens."""
    at = [(c.rows(s, torch.arange(t)), torch.arange(t, device=c.dev)) for s, t in enumerate(c.total)]
    return torch.cat([r for r, _ in at]), torch.cat([p for _, p in at])


def _cancelling(new, total, nq, nkv, dev="cuda"):
    """bf16: of each granule's keys eight have the weight 1 and the value -1, eight a
    weight just under 0.5 (1 + 2^-8), which 8 bits hold as 0.5, and the value 2."""
    c = Case(900 + new, "bf16", [new, new], [total, max(new, total // 3)], nq=nq, nkv=nkv, dev=dev)
    c.q.zero_()
    c.q[..., :2] = 1.0
    rows, pos = _held(c)
    light = (pos % 16 >= 8)[:, None]
    y = math.log(0.5 * (1 + 0.98 * 2.0 ** -8))
    hi = float(torch.tensor(y).bfloat16())
    k = torch.zeros(len(rows), nkv, D, device=c.dev)
    k[..., 0] = torch.where(light, hi, 0.0)
    k[..., 1] = torch.where(light, y - hi, 0.0)
    c.k[rows] = k.bfloat16()
    c.v[rows] = torch.where(light[..., None], 2.0, -1.0).expand(-1, nkv, D).bfloat16()
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("new,total,nq,nkv", [(1, 16, 32, 4), (1, 2000, 32, 4), (2, 333, 32, 4),
                                              (1, 40000, 8, 1), (8, 700, 8, 4)])
def test_sixteen_bits_of_a_weight_in_bf16_next_tokens(m, ws, new, total, nq, nkv):
    c = _cancelling(new, total, nq, nkv)
    c.check(c.attend(m, ws, scale=1.0), scale=1.0, p_bits=16)


def test_eight_bits_would_be_found():
    """The same inputs on the CPU with weights rounded to bf16: beyond the tolerance."""
    c = _cancelling(1, 333, 4, 2, dev="cpu")
    ref, tol = c.reference(scale=1.0, p_bits=16)
    kd, vd = c.k.double(), c.v.double()
    for s, total in enumerate(c.total):
        rows = c.rows(s, torch.arange(total))
        p = torch.exp(kd[rows, 0, :2].sum(1))
        for bits, inside in ((p, True), (p.bfloat16().double(), False)):
            out = (bits[:, None] * vd[rows, 0]).sum(0) / p.sum()
            off = (out.bfloat16().double() - ref[s, 0]).abs()
            assert bool((off <= tol[s, 0]).all()) is inside


@pytest.mark.gpu
@pytest.mark.parametrize("heavy", ["each granule", "the first key"])
@pytest.mark.parametrize("new,nq,nkv", [(1, 32, 4), (2, 32, 4), (20, 32, 4), (70, 4, 4)])
@pytest.mark.parametrize("total", [90, 5000])
def test_small_weights_beside_a_large_one_in_e4m3(m, ws, heavy, new, nq, nkv, total):
    """Keys of the weight e^-18 = 2^-25.97 beside keys of the weight 1 whose values
    are zero: the outputs are the small weights' alone.  A weight is held in f16
    relative to 2^-7 of the largest, in steps of 2^-24 of that: off by half a step,
    2^-32 of the largest, a key; scores are exact, the exponent's argument is good to
    2^-19, sums to 2^-17, and one rounding to bf16 (2^-8) is at the end."""
    c = Case(910 + new, "e4m3", [new], [total], nq=nq, nkv=nkv)
    c.q.zero_()
    c.q[..., 0] = 1.0
    rows, pos = _held(c)
    big = pos % 16 == 0 if heavy == "each granule" else pos == 0
    g = torch.Generator("cuda").manual_seed(77)
    k = torch.zeros(len(rows), nkv, D, device="cuda")
    k[..., 0] = torch.where(big, 0.0, -18.0)[:, None]
    v = 128.0 + 128.0 * torch.rand(len(rows), nkv, D, generator=g, device="cuda")
    v[big] = 0.0
    c.k[rows] = k.to(torch.float8_e4m3fn).view(torch.uint8)
    c.v[rows] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    c.ks[rows // BLOCK], c.vs[rows // BLOCK] = 1.0, 2.0 ** -8
    got = c.attend(m, ws, scale=1.0).double()
    w = torch.where(big, 1.0, math.exp(-18.0)).double()
    v = c.value(c.v, c.vs)[rows]
    seen = (pos[None] <= torch.arange(total - new, total, device="cuda")[:, None]).double()
    den = (seen * w).sum(1)[:, None, None]
    ref = torch.einsum("tj,jhd->thd", seen * w, v) / den
    half_steps = 2.0 ** -32 * torch.einsum("tj,jhd->thd", seen, v) / den
    ref, half_steps = (x.repeat_interleave(nq // nkv, 1) for x in (ref, half_steps))
    off = (got - ref).abs() - ref * (2.0 ** -8 + 2.0 ** -15) - half_steps - 1e-35
    assert float(off.max()) <= 0.0, (float(off.max()), float(ref.max()), got.flatten()[:4].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 2, 24])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -40])
def test_scales_of_zero(m, ws, new, scale):
    """A cache of zeros with scales of zero beside blocks of the smallest scale, or
    alone: finite, and the keys count in the denominator.  (No append writes a scale
    of zero; it counts as 2^-80, so that the one code, 1.0, is there as 2^-80 / seen,
    rounded as any output is: to bf16, 2^-8 of it, the rest fp32, within 2^-7.)"""
    c = Case(920 + new, "e4m3", [new], [2000])
    rows, pos = _held(c)
    c.k[rows] = 0
    c.v[rows] = 0
    c.ks[rows // BLOCK], c.vs[rows // BLOCK] = 0.0, 0.0
    last = pos >= 1984
    c.vs[rows[last] // BLOCK] = scale
    c.v[rows[pos == 1984]] = 0x38     # 1.0
    got = c.attend(m, ws).double()
    seen = torch.arange(2001 - new, 2001, device="cuda").double()
    ref = (torch.arange(2000 - new, 2000, device="cuda") >= 1984).double() * scale / seen
    off = (got - ref[:, None, None]).abs()
    assert (off <= ref[:, None, None] * 2.0 ** -7 + (1 + 2.0 ** -7) * 2.0 ** -80 / seen[:, None, None]).all()

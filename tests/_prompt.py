"""Plain 64-bit forms of the linear side of a prompt, and how far a kernel may be from them."""
from __future__ import annotations

import torch

import moe_decode_sigmoid_gb300 as m

NONE, SILU, GELU, SWIGLU = m.FLINT_ACT_NONE, m.FLINT_ACT_SILU, m.FLINT_ACT_GELU, m.FLINT_ACT_SWIGLU
# A product of n_in terms in fp32, the terms themselves exact (two 8-bit significands): n_in
# additions, each off by at most one unit of the last place, 2^-23, of the sum of the terms'
# sizes (tensor cores may cut instead of rounding); and a few more for bias and splits.
ADD = 2.0 ** -23


def gen(seed, dev="cuda"):
    return torch.Generator(dev).manual_seed(seed)


def bf(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * scale).bfloat16()


def _act(y, err, act):
    """(act(y), how far it may be off for sums off by err).  Slopes: silu below 1.1, gelu
    below 1.13; the activation's own fp32 arithmetic within 16 half steps of its value."""
    own = 16 * 2.0 ** -24
    if act == SWIGLU:
        n = y.shape[1] // 2
        (g, u), (eg, eu) = (y[:, :n], y[:, n:]), (err[:, :n], err[:, n:])
        s = g * torch.sigmoid(g)
        es = 1.1 * eg + own * s.abs()
        return s * u, es * (u.abs() + eu) + s.abs() * eu + own * (s * u).abs()
    if act == SILU:
        s = y * torch.sigmoid(y)
        return s, 1.1 * err + own * s.abs()
    if act == GELU:
        s = 0.5 * y * torch.special.erfc(-y * 0.5 ** 0.5)
        return s, 1.13 * err + own * s.abs()
    return y, err


def linear(x, w, bias, residual, act, dtype):
    """(64-bit values, how far an output may be from each)."""
    x, w = x.double(), w.double()
    y, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    y, err = _act(y, (x.shape[1] + 16) * ADD * size, act)
    if residual is not None:
        y = y + residual.double()
        err = err + 2.0 ** -24 * (y.abs() + residual.double().abs())
    # the output's own rounding: half a step, of a value that may be off itself; the
    # smallest normal number for what falls below it
    half = torch.finfo(dtype).eps / 2
    return y, err + half * (y.abs() + err) + torch.finfo(dtype).tiny


def check(got, want, name=""):
    y, err = want
    got = got.double()
    assert torch.isfinite(got).all(), name
    off = (got - y).abs() - err
    i = int(off.argmax())
    assert off.flatten()[i] <= 0, "%s: %g where %g is right, %g allowed" % (
        name, got.flatten()[i], y.flatten()[i], err.flatten()[i])


def grouped(x, w, start, index, bias, act, dtype, rows):
    """(rows that a group has, 64-bit values, errors), row by row in group order."""
    start = [min(max(int(s), 0), rows) for s in start]
    out = {}
    for g in range(w.shape[0]):
        r = list(range(start[g], max(start[g], start[g + 1])))
        if index is not None:
            r = [i for i in r if 0 <= int(index[i]) < x.shape[0]]
        if r:
            src = x[[int(index[i]) for i in r]] if index is not None else x[r]
            y, err = linear(src, w[g], None if bias is None else bias[g], None, act, dtype)
            out.update({i: (y[k], err[k]) for k, i in enumerate(r)})
    return out


def choose(logits, offset, select_only, k=6):
    """(experts in rank order, weights) in 64 bits; equal keys: the lower index."""
    key = logits if offset is None else (logits + offset)   # fp32, as the definition says
    order = torch.sort(torch.nan_to_num(key.double(), nan=1e300, posinf=1e299, neginf=-1e299), dim=1,
                       descending=True, stable=True).indices[:, :k]
    s = torch.sigmoid((logits if select_only else key).double().gather(1, order))
    total = s.sum(1, keepdim=True)
    return order, torch.where(total == 0, torch.zeros_like(s), s / total)


def order_of(idx, n_experts=256):
    """(start, token of each row, row of each pair) of the stable order by expert."""
    flat = idx.flatten().long()
    pair = torch.sort(flat, stable=True).indices
    row = torch.empty_like(pair)
    row[pair] = torch.arange(pair.numel(), device=idx.device)
    start = torch.zeros(n_experts + 1, dtype=torch.int64, device=idx.device)
    start[1:] = torch.bincount(flat, minlength=n_experts).cumsum(0)
    return start, pair // idx.shape[1], row.view(idx.shape)

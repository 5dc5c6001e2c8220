"""Paged KV-cache cases and their plain 64-bit values (torch float64, on the
device the case lives on), for the tests of the paged append and attention."""
from __future__ import annotations

import math

import torch

D = 128
BLOCK = 16
LOG2E = 1.4426950408889634


def pages_for(total, page, extra, gen, dev, max_pages=None, dead=-1):
    """(page table, pages of the cache): every sequence's pages at random
    places, `dead` in the entries behind them."""
    need = [max(0, -(-t // page)) for t in total]
    n_pages = sum(need) + extra
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    cols = max_pages or max(1, max(need))
    table = torch.full((len(total), cols), dead, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table.to(dev), n_pages


class Case:
    """Sequences with new[s] rows and total[s] tokens; the cache rows that hold
    tokens 0 .. total[s] - 1 have values, all others garbage (NaN)."""

    def __init__(self, seed, fmt, new, total, page=16, nq=32, nkv=4, dev="cuda", extra=2, rows_after=0,
                 loud=1.0, max_pages=None, dead=-1, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.new, self.total, self.page, self.nq, self.nkv = fmt, new, total, page, nq, nkv
        self.dev = torch.device(dev)
        self.n = len(new)
        start = [0]
        for x in new:
            start.append(start[-1] + x)
        self.start, self.T = start, start[-1] + rows_after
        self.q_start = torch.tensor(start, dtype=torch.int32, device=dev)
        self.kv_len = torch.tensor(total, dtype=torch.int32, device=dev)
        self.table, self.n_pages = pages_for(total, page, extra, g, dev, max_pages, dead)
        rows = self.n_pages * page
        dg = torch.Generator(dev).manual_seed(seed + 1)
        self.q = (size * torch.randn(self.T, nq, D, generator=dg, device=dev)).to(torch.bfloat16)
        self.sinks = torch.randn(nq, generator=dg, device=dev)

        def cache(size):
            x = torch.randn(rows, nkv, D, generator=dg, device=dev) * size
            x *= torch.exp(loud * torch.randn(rows, nkv, 1, generator=dg, device=dev))
            if fmt == "bf16":
                return x.to(torch.bfloat16), None
            amax = x.view(-1, BLOCK, nkv, D).abs().amax(dim=(1, 3))
            s = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
            c = (x.view(-1, BLOCK, nkv, D) / s[:, None, :, None]).clamp(-448, 448)
            return c.to(torch.float8_e4m3fn).view(rows, nkv, D).view(torch.uint8), s

        (self.k, self.ks), (self.v, self.vs) = cache(size), cache(1.0)
        held = torch.zeros(rows, dtype=torch.bool, device=dev)
        for s in range(self.n):
            if total[s] > 0:
                held[self.rows(s, torch.arange(total[s]))] = True
        for c, sc in ((self.k, self.ks), (self.v, self.vs)):
            if fmt == "bf16":
                c[~held] = float("nan")
            else:
                c[~held] = 0x7F
                sc[~held.view(-1, BLOCK).any(1)] = float("nan")

    def rows(self, s, pos):
        t = self.table[s].cpu().long()
        return (t[pos // self.page] * self.page + pos % self.page).to(self.dev)

    def shaped(self, c):
        return c.view(self.n_pages, self.page, self.nkv, D)

    def scaled(self, sc):
        return sc.view(self.n_pages, self.page // BLOCK, self.nkv)

    def value(self, c, sc):
        """The cache's rows as float64."""
        if self.fmt == "bf16":
            return c.double()
        x = c.view(torch.float8_e4m3fn).double().view(-1, BLOCK, self.nkv, D)
        return (x * sc.double()[:, None, :, None]).view(-1, self.nkv, D)

    def batch(self, m, max_q=None):
        return m.PagedBatch(self.q_start, self.kv_len, self.table, self.page,
                            max_q or max(1, max(self.new)))

    def attend(self, m, ws, window=0, sinks=None, scale=None, max_q=None, out=None, stream=None,
               batch=None):
        out = torch.full_like(self.q, 7.25) if out is None else out
        b = batch or self.batch(m, max_q)
        dims = m.AttnDims(self.nq, self.nkv, D)
        if self.fmt == "bf16":
            m.flint_attn_paged_bf16(self.q, self.shaped(self.k), self.shaped(self.v), b, out, ws,
                                    sinks=sinks, window=window, softmax_scale=scale, dims=dims,
                                    stream=stream)
        else:
            m.flint_attn_paged_fp8(self.q, self.shaped(self.k), self.shaped(self.v),
                                   self.scaled(self.ks), self.scaled(self.vs), b, out, ws,
                                   sinks=sinks, window=window, softmax_scale=scale, dims=dims,
                                   stream=stream)
        return out

    def reference(self, window=0, sinks=None, scale=None, absent=(), p_bits=None):
        """(values, tolerances) of the attention's rows, float64 [T, nq, D]; rows
        that no sequence brings are NaN in both.  absent: (sequence, page) pairs
        the table does not hold.

        Tolerance of an output element, with p_j the exact weights, A = sum p_j
        |v_j| over the denominator and S the largest sum of |q_d k_jd| scale:
          - one rounding to bf16: 2^-8 of the value;
          - a score is a dot product of 128 terms in fp32: 128 2^-24 S off at
            most, and the exponent's argument 2^-21 S more; e^s is off by as
            much, in the numerator and the denominator;
          - over an E4M3 cache a query's elements count to 2^-18 of its largest:
            F = 2^-18 max |q_d| sum |k_jd| scale at most in a score;
          - the weights enter the second product with p_bits significant bits
            (rounded: 2^-p_bits), and, as f16, with an absolute step of 2^-24 of
            the largest weight-times-scale (half of it is charged for each key);
          - fp32 sums over n keys, at most n / 16 + 64 additions deep."""
        scale = D ** -0.5 if scale is None else scale
        if p_bits is None:
            p_bits = 11 if self.fmt == "e4m3" else 8
        kd, vd = self.value(self.k, self.ks), self.value(self.v, self.vs)
        out = torch.full((self.T, self.nq, D), float("nan"), dtype=torch.float64, device=self.dev)
        tol = out.clone()
        g = self.nq // self.nkv
        for s in range(self.n):
            n, total = self.new[s], self.total[s]
            if n == 0:
                continue
            sl = slice(self.start[s], self.start[s + 1])
            if total == 0:
                out[sl], tol[sl] = 0.0, 0.0
                continue
            keys = torch.arange(total)
            keep = torch.ones(total, dtype=torch.bool)
            for (ss, page) in absent:
                if ss == s:
                    keep[page * self.page:(page + 1) * self.page] = False
            pos = torch.arange(total - n, total)
            low = max(0, int(pos[0]) - window + 1) if window else 0
            keep[:low] = False
            keys = keys[keep]
            if len(keys) == 0:
                out[sl], tol[sl] = 0.0, 0.0
                continue
            rows = self.rows(s, keys)
            k, v = kd[rows], vd[rows]
            keys, pos = keys.to(self.dev), pos.to(self.dev)
            hide = keys[None] > pos[:, None]
            if window:
                hide |= keys[None] <= pos[:, None] - window
            for h in range(self.nq):
                q = self.q[sl, h].double()
                sc = (q @ k[:, h // g].T) * scale
                big = float((q.abs() @ k[:, h // g].abs().T).max()) * scale
                flat = 0.0
                if self.fmt == "e4m3":
                    flat = float(q.abs().max() * k[:, h // g].abs().nan_to_num(0.0).sum(1).max()) * scale
                sc = sc.masked_fill(hide, -math.inf)
                top = sc.amax(1, keepdim=True)
                if sinks is not None:
                    top = torch.maximum(top, sinks[h].double())
                top = torch.where(top == -math.inf, torch.zeros_like(top), top)
                p = torch.exp(sc - top)
                den = p.sum(1, keepdim=True)
                if sinks is not None:
                    den = den + torch.exp(sinks[h].double() - top)
                seen = (~hide).any(1, keepdim=True)
                p = torch.where(seen, p / den, torch.zeros_like(p))
                vh = torch.where(v[:, h // g].isnan(), torch.zeros_like(v[:, h // g]), v[:, h // g])
                out[sl, h] = p @ vh
                mass = p @ vh.abs()
                nk = len(keys)
                c = 2 * (2.0 ** -17 + 2.0 ** -21) * big + 2 * 2.0 ** -18 * flat + 2.0 ** -p_bits + 2.0 ** -21 + \
                    2.0 ** -23 * (nk / 16 + 64)
                low_p = 0.0
                if self.fmt == "e4m3":
                    vs = self.vs.double()[rows // BLOCK, h // g]
                    low_p = nk * 2.0 ** -25 * 448 * (p * vs[None]).amax(1, keepdim=True)
                tol[sl, h] = 2.0 ** -8 * out[sl, h].abs() + c * mass + low_p + 1e-35
        return out, tol

    def check(self, got, window=0, sinks=None, scale=None, absent=(), p_bits=None):
        ref, tol = self.reference(window, sinks, scale, absent, p_bits)
        used = ~ref[:, 0, 0].isnan()
        off = (got[used].double() - ref[used]).abs() - tol[used]
        assert not got[used].isnan().any()
        assert float(off.max()) <= 0.0, (float(off.max()), torch.nonzero(off > 0)[:5].tolist(),
                                         float((off > 0).double().mean()))
        assert (got[~used] == 7.25).all()


def append_reference(qkv, q_norm, k_norm, pos, nq, nkv, theta, eps):
    """(q, k, v, bounds of |q|'s and |k|'s fp32 error) in float64.

    The norm is a product of a 128-term fp32 sum's root and two factors: 2^-17
    of the value covers it; an angle reduced to [-pi, pi] is held in fp32 (2^-22)
    and its sine and cosine are good to 2^-22, so a turned element is off by at
    most 2^-17 of |a| + |b|."""
    x = qkv.double().view(qkv.shape[0], -1, D)
    res = []
    for part, g in ((x[:, :nq], q_norm), (x[:, nq:nq + nkv], k_norm)):
        y = part / (part.square().mean(-1, keepdim=True) + eps).sqrt() * g.double()
        size = y.abs()
        if theta > 0:
            f = theta ** (-torch.arange(D // 2, dtype=torch.float64, device=y.device) * 2 / D)
            a = pos.double()[:, None, None] * f
            c, s = a.cos(), a.sin()
            lo, hi = y[..., :64], y[..., 64:]
            y = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
            size = (lo.abs() + hi.abs()).repeat(1, 1, 2)
        res.append((y, size * 2.0 ** -17))
    return res[0][0], res[1][0], x[:, nq + nkv:], res[0][1], res[1][1]

"""GPU parity of the paged append (Q/K norm + RoPE + cache write), of its E4M3
quantisation, and of append and attention run together as a decode loop."""
from __future__ import annotations

import pytest
import torch

from tests._paged import BLOCK, Case, D, append_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    import moe_decode_sigmoid_gb300 as mod
    mod.lib()
    return mod


def _rows(c, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    qkv = (size * torch.randn(c.T, (c.nq + 2 * c.nkv) * D, generator=g, device="cuda")).to(torch.bfloat16)
    gains = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    return qkv, gains[0], gains[1]


def _append(m, c, qkv, qn, kn, theta, eps=1e-6, batch=None, q=None):
    q = torch.full_like(c.q, 7.25) if q is None else q
    dims = m.AttnDims(c.nq, c.nkv, D)
    b = batch or c.batch(m)
    if c.fmt == "bf16":
        m.flint_qk_norm_rope_kv_paged_bf16(qkv, qn, kn, b, q, c.shaped(c.k), c.shaped(c.v), theta, eps,
                                           dims=dims)
    else:
        m.flint_qk_norm_rope_kv_paged_fp8(qkv, qn, kn, b, q, c.shaped(c.k), c.shaped(c.v),
                                          c.scaled(c.ks), c.scaled(c.vs), theta, eps, dims=dims)
    return q


def _check_append(c, qkv, qn, kn, theta, eps, q, before, gone=()):
    """Against 64 bits: one bf16 rounding (2^-8 of the value) or one E4M3
    rounding (2^-4, at least half a subnormal step 2^-10) over the fp32 error;
    every row that nothing was appended to bit for bit as before."""
    k0, v0, ks0, vs0 = before
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(c.new, c.total)]).cuda()
    used = c.start[-1]
    qr, kr, vr, qe, ke = append_reference(qkv[:used], qn, kn, pos, c.nq, c.nkv, theta, eps)
    assert ((q[:used].double() - qr).abs() <= 2.0 ** -8 * qr.abs() + qe + 1e-30).all()
    assert (q[used:] == 7.25).all()
    same = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")
    same_scale = torch.ones(c.k.shape[0] // BLOCK, dtype=torch.bool, device="cuda")
    for s in range(c.n):
        n, total = c.new[s], c.total[s]
        p = torch.arange(max(0, total - n), total)
        if len(p) == 0:
            continue
        there = torch.ones(len(p), dtype=torch.bool)
        for (ss, page) in gone:
            if ss == s:
                there &= p // c.page != page
        t = c.start[s] + p - (total - n)
        p, t = p[there], t[there]
        if len(p) == 0:
            continue
        rows = c.rows(s, p)
        same[rows] = False
        t = t.cuda()
        if c.fmt == "bf16":
            assert ((c.k[rows].double() - kr[t]).abs() <= 2.0 ** -8 * kr[t].abs() + ke[t] + 1e-30).all()
            want = qkv[t].view(len(t), -1, D)[:, c.nq + c.nkv:]
            assert torch.equal(c.v[rows].view(torch.int16), want.view(torch.int16))
            continue
        for cache, scale, old, old_scale, x, err in ((c.k, c.ks, k0, ks0, kr[t], ke[t]),
                                                     (c.v, c.vs, v0, vs0, vr[t], 0 * vr[t])):
            blocks = (rows // BLOCK).unique()
            same_scale[blocks] = False
            for b in blocks.tolist():
                at = (rows // BLOCK == b).nonzero()[:, 0]
                amax = x[at].abs().amax(dim=(0, 2))
                off = err[at].abs().amax()
                lo, hi = ((amax + o).clamp(min=448 * 2.0 ** -40).div(448).log2().ceil().clamp(-40, 40).exp2()
                          for o in (-off, off))
                kept = int(p[at[0].item()]) % BLOCK
                if kept:
                    lo, hi = (torch.maximum(v, old_scale[b].double()) for v in (lo, hi))
                got = scale[b].double()
                assert ((got == lo) | (got == hi)).all(), (got, lo, hi)
                code = cache[rows[at]].view(torch.float8_e4m3fn).double()
                want = (x[at] / got[:, None]).clamp(-448, 448)
                bound = 2.0 ** -4 * want.abs() + 2.0 ** -10 + err[at] / got[:, None]
                assert ((code - want).abs() <= bound).all()
                if kept:
                    r = slice(b * BLOCK, b * BLOCK + kept)
                    same[r] = False
                    had = old[r].view(torch.float8_e4m3fn).double()
                    now = cache[r].view(torch.float8_e4m3fn).double()
                    ratio = (old_scale[b].double() / got)[None, :, None]
                    want = had * ratio
                    grew = (ratio < 1).expand_as(had)
                    assert ((now - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10)[grew].all()
                    exact = grew & (want.abs() >= 2.0 ** -6)
                    assert (now == want)[exact].all()
                    assert torch.equal(cache[r][~grew], old[r][~grew])
    assert torch.equal(c.k[same].view(torch.uint8), k0[same].view(torch.uint8))
    assert torch.equal(c.v[same].view(torch.uint8), v0[same].view(torch.uint8))
    if c.fmt == "e4m3":
        for a, b in ((c.ks, ks0), (c.vs, vs0)):
            assert torch.equal(a[same_scale].view(torch.int32), b[same_scale].view(torch.int32))


def _kept(c):
    return [None if x is None else x.clone() for x in (c.k, c.v, c.ks, c.vs)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total,page,theta", [
    ([1], [1], 16, 1e6), ([1], [16], 16, 1e6), ([1], [17], 16, 0.0), ([1] * 9, [3, 900, 31, 32, 33, 1, 64, 5, 77], 32, 1e6),
    ([16], [16], 16, 1e6), ([40], [40], 16, 1e4), ([33, 0, 2, 100], [50, 7, 2, 1111], 64, 1e6),
    ([500], [200000], 128, 1e6), ([3] * 60, [40] * 60, 16, 0.0)])
def test_append(m, fmt, new, total, page, theta):
    c = Case(301 + len(new) + new[0], fmt, new, total, page=page, rows_after=3)
    rows = _rows(c, 401)
    before = _kept(c)
    q = _append(m, c, *rows, theta)
    _check_append(c, *rows, theta, 1e-6, q, before)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (8, 8), (4, 2), (64, 8), (2, 1), (16, 4)])
def test_append_head_layouts(m, fmt, nq, nkv):
    c = Case(311, fmt, [5, 1, 40], [9, 30, 47], nq=nq, nkv=nkv)
    rows = _rows(c, 402)
    before = _kept(c)
    q = _append(m, c, *rows, 1e6)
    _check_append(c, *rows, 1e6, 1e-6, q, before)


@pytest.mark.parametrize("size", [1e-30, 1e-5, 300.0, 1e15])
def test_block_scales_follow_the_values(m, size):
    """Values far above and below the block's earlier ones: scales grow and the
    earlier codes are rewritten, or stay; at the ends they are clamped."""
    c = Case(312, "e4m3", [1, 4, 20], [25, 13, 33])
    rows = _rows(c, 403, size)
    before = _kept(c)
    q = _append(m, c, *rows, 1e6, 0.25)
    _check_append(c, *rows, 1e6, 0.25, q, before)


def test_zeros_infinities_and_nan(m):
    c = Case(313, "e4m3", [20], [20])
    qkv, qn, kn = _rows(c, 404)
    v = qkv.view(c.T, -1, D)[:, c.nq + c.nkv:]
    v[:16, 0] = 0.0                      # a head whose block is all zeros
    v[3, 1, 5] = float("inf")
    v[4, 1, 6] = float("-inf")
    v[5, 1, 7] = float("nan")
    _append(m, c, qkv, qn, kn, 1e6)
    r = c.rows(0, torch.arange(16))
    b = int(r[0]) // BLOCK
    code = c.v[r].view(torch.float8_e4m3fn).float()
    assert (code[:, 0] == 0).all() and float(c.vs[b, 0]) == 2.0 ** -40
    assert code[3, 1, 5] == 448 and code[4, 1, 6] == -448 and code[5, 1, 7].isnan()
    rest = v[:16, 1].float()
    rest = rest[rest.isfinite()].abs().max()
    assert float(c.vs[b, 1]) == float(torch.exp2(torch.ceil(torch.log2(rest / 448))))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_rows_that_have_no_place(m, fmt):
    """Pages outside the cache, and rows before the cache's start, write nothing;
    their queries are still normed and turned."""
    c = Case(314, fmt, [70, 6, 1], [100, 4, 20], page=32)
    c.table[0, 2] = 0
    table = c.table.clone()
    table[0, 2] = c.n_pages
    table[2, 0] = -1
    rows = _rows(c, 405)
    before = _kept(c)
    b = m.PagedBatch(c.q_start, c.kv_len, table, c.page, 70)
    q = _append(m, c, *rows, 1e6, batch=b)
    _check_append(c, *rows, 1e6, 1e-6, q, before, gone=[(0, 2), (2, 0)])


def test_the_bf16_rows_are_the_slot_calls(m):
    """A decode step's rows through flint_qk_norm_rope_kv_bf16 with the slots the
    page table gives, and through the paged call: the same values."""
    c = Case(315, "bf16", [1] * 7, [5, 900, 33, 32, 31, 1, 64], page=32)
    qkv, qn, kn = _rows(c, 406)
    k1, v1 = c.k.clone(), c.v.clone()
    q = _append(m, c, qkv, qn, kn, 1e6)
    slots = torch.stack([c.rows(s, torch.tensor([t - 1]))[0] for s, t in enumerate(c.total)])
    q1 = torch.empty_like(q)
    m.flint_qk_norm_rope_kv_bf16(qkv, qn, kn, (c.kv_len - 1).contiguous(), slots.to(torch.int32), q1,
                                 k1, v1, 1e6)
    assert torch.equal(c.v.view(torch.int16), v1.view(torch.int16))
    # two orders of an fp32 sum: at most one bf16 step apart (2^-7 of the value)
    held = ~c.k.isnan()
    for a, b in ((q, q1), (c.k[held], k1[held])):
        assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 2.0 ** -14).all()


def test_batch_with_hostile_numbers_stays_in_bounds(m):
    c = Case(316, "e4m3", [4, 4], [100, 60], rows_after=2)
    rows = _rows(c, 407)
    guard = torch.full((c.T + 64, c.nq, D), 7.25, dtype=torch.bfloat16, device="cuda")
    for q_start, kv in (([0, 4, 1 << 30], [100, 60]), ([-5, 4, 5], [100, 1 << 30]),
                        ([4, 0, -3], [-9, 60]), ([0, (1 << 31) - 1, 0], [-(1 << 31), 60])):
        b = m.PagedBatch(torch.tensor(q_start, dtype=torch.int32, device="cuda"),
                         torch.tensor(kv, dtype=torch.int32, device="cuda"), c.table, c.page, 4)
        _append(m, c, *rows, 1e6, batch=b, q=guard[32:32 + c.T])
    torch.cuda.synchronize()
    assert (guard[:32] == 7.25).all() and (guard[32 + c.T:] == 7.25).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, False), (40, True)])
def test_prompt_then_decode_as_it_would_be_used(m, fmt, window, sinks):
    """A prompt appended and attended in two chunks, then decode steps replayed
    from one captured graph that refills lengths and rows in place, all over
    one cache: each attention against 64 bits on the cache as it then is."""
    c = Case(317, fmt, [30, 50], [30, 50], page=32, max_pages=6, extra=8)
    table = c.table.clone()
    free = [p for p in range(c.n_pages) if p not in set(c.table.flatten().tolist())]
    for s in range(2):
        have = int((table[s] >= 0).sum())
        while have < 4:
            table[s, have] = free.pop()
            have += 1
    c.table.copy_(table)
    for x in (c.k, c.v):
        x.copy_(torch.full_like(x, float("nan")) if fmt == "bf16" else torch.full_like(x, 0x7F))
    ws = m.new_attn_workspace()
    sk = c.sinks if sinks else None
    done = [0, 0]
    for chunk in ([30, 50], [17, 1]):
        c.new, c.total = chunk, [d + n for d, n in zip(done, chunk)]
        done = c.total
        c.start = [0, chunk[0], sum(chunk)]
        c.T = sum(chunk)
        c.q_start.copy_(torch.tensor(c.start, dtype=torch.int32))
        c.kv_len.copy_(torch.tensor(c.total, dtype=torch.int32))
        c.q = torch.empty(c.T, c.nq, D, dtype=torch.bfloat16, device="cuda")
        rows = _rows(c, 408 + c.T)
        before = _kept(c)
        c.q = _append(m, c, *rows, 1e6)
        _check_append(c, *rows, 1e6, 1e-6, c.q, before)
        c.check(c.attend(m, ws, window, sk), window, sk)
    c.new, c.start, c.T = [1, 1], [0, 1, 2], 2
    c.q_start.copy_(torch.tensor(c.start, dtype=torch.int32))
    c.q = torch.empty(2, c.nq, D, dtype=torch.bfloat16, device="cuda")
    qkv, qn, kn = _rows(c, 500)
    out = torch.full_like(c.q, 7.25)
    b = c.batch(m, 1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _append(m, c, qkv, qn, kn, 1e6, batch=b, q=c.q)
        c.attend(m, ws, window, sk, batch=b, out=out)
    for step in range(20):
        c.total = [d + 1 for d in done]
        done = c.total
        c.kv_len.copy_(torch.tensor(c.total, dtype=torch.int32))
        qkv.copy_(_rows(c, 600 + step, 1.5 ** step)[0])
        before = _kept(c)
        graph.replay()
        torch.cuda.synchronize()
        _check_append(c, qkv, qn, kn, 1e6, 1e-6, c.q, before)
        c.check(out, window, sk)

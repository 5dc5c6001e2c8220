"""GPU parity of the paged attention where a few rows a sequence share the
next-token kernel, where one row is joined from many parts, and in the uses a
program makes of it: shared workspaces, shared pages, other devices' streams.
Tolerances: tests/_paged.py."""
from __future__ import annotations

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


@pytest.fixture(scope="module")
def ws(m):
    return m.new_attn_workspace()


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv,q", [(32, 4, 2), (16, 4, 4), (16, 4, 3), (8, 4, 5), (8, 4, 8),
                                      (4, 4, 8), (4, 4, 9), (4, 4, 16), (8, 1, 2), (64, 8, 2)])
@pytest.mark.parametrize("window,sinks", [(0, False), (19, True)])
def test_few_rows_a_sequence(m, ws, fmt, nq, nkv, q, window, sinks):
    """Up to 16 rows a KV head, sequences of fewer rows than others and of none,
    lengths around a granule's and a window's edge."""
    new = [q, 1, 0, max(1, q - 1), q, q]
    total = [1000, 17, 5, 16 + q - 1, q, 33]
    c = Case(300 + nq + q, fmt, new, total, page=16, nq=nq, nkv=nkv, rows_after=3)
    s = c.sinks if sinks else None
    c.check(c.attend(m, ws, window, s), window, s)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv,new,total", [
    (8, 1, 1, 66001), (8, 1, 2, 66001), (8, 1, 5, 30011), (8, 1, 16, 20000), (8, 1, 40, 20000),
    (4, 4, 13, 30000), (2, 2, 200, 9000)])
def test_one_sequence_over_all_ctas(m, ws, fmt, nq, nkv, new, total):
    """Rows cut into up to 152 parts, joined in two steps; then a short call on
    the same workspace, whose counters have to be back at zero."""
    c = Case(320 + new, fmt, [new], [total], page=64, nq=nq, nkv=nkv)
    first = c.attend(m, ws, 0, c.sinks)
    c.check(first, 0, c.sinks)
    assert same(c.attend(m, ws, 0, c.sinks), first)
    d = Case(321, fmt, [1, 3], [300, 4000])
    d.check(d.attend(m, ws))
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv", [(8, 1), (4, 4)])
@pytest.mark.parametrize("q", [1, 2, 30])
def test_the_widest_window_and_rows_before_the_start(m, ws, fmt, nq, nkv, q):
    c = Case(330, fmt, [q, q], [300, max(0, q - 1)], nq=nq, nkv=nkv)
    wide = (1 << 31) - 1
    got = c.attend(m, ws, wide, c.sinks)
    c.check(got, 0, c.sinks)
    assert same(got, c.attend(m, ws, 0, c.sinks))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_the_most_rows_and_sequences(m, ws, fmt):
    """8192 rows of 256 sequences: every item list and table at its largest."""
    for nq, nkv, new in ((8, 1, [32] * 256), (8, 1, [1] * 255 + [8192 - 255]), (2, 2, [31, 33] * 128)):
        c = Case(340, fmt, new, [n + 40 for n in new], nq=nq, nkv=nkv)
        c.check(c.attend(m, ws, 50), 50)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 2, 24])
def test_sequences_that_share_pages(m, ws, fmt, new):
    """A prompt's pages read by two sequences, and by one of them twice."""
    c = Case(350, fmt, [new, new], [640, 640], page=64)
    table = c.table.clone()
    table[1, :6] = table[0, :6]
    table[1, 3] = table[1, 2]
    c.table = table
    c.check(c.attend(m, ws))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_two_captured_graphs_share_a_workspace(m, ws, fmt):
    cases = [Case(360, fmt, [1] * 3, [30000, 17, 5000], nq=8, nkv=1),
             Case(361, fmt, [70, 2], [9000, 20000], nq=8, nkv=1)]
    alone = [c.attend(m, ws) for c in cases]
    outs = [torch.full_like(a, 7.25) for a in alone]
    graphs = []
    for c, o in zip(cases, outs):
        b = c.batch(m)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.attend(m, ws, out=o, batch=b)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.fill_(7.25)
            g.replay()
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert same(a, o)
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q", [2, 24])
def test_draft_rows_equal_next_tokens_one_by_one(m, ws, fmt, q):
    """The row of a drafted token sees what the same token sees when it is the
    newest, so both lie within the tolerance of the same value; rows behind it
    in the cache, NaN included, change nothing."""
    c = Case(370, fmt, [q, q], [100 + q, 40 + q], nq=8, nkv=2)
    ref, tol = c.reference()
    for i in range(q):
        one = torch.stack([c.q[i], c.q[q + i]])
        out = torch.empty_like(one)
        b = m.PagedBatch(torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"),
                         c.kv_len - (q - 1 - i), c.table, c.page, 1)
        dims = m.AttnDims(8, 2, D)
        if fmt == "bf16":
            m.flint_attn_paged_bf16(one, c.shaped(c.k), c.shaped(c.v), b, out, ws, dims=dims)
        else:
            m.flint_attn_paged_fp8(one, c.shaped(c.k), c.shaped(c.v), c.scaled(c.ks),
                                   c.scaled(c.vs), b, out, ws, dims=dims)
        at = [i, q + i]
        assert ((out.double() - ref[at]).abs() <= tol[at]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_q", [1 << 29, (1 << 31) - 1])
def test_any_bound_on_new_tokens(m, ws, fmt, max_q):
    c = Case(380, fmt, [20, 1], [300, 90])
    c.check(c.attend(m, ws, max_q=max_q))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total", [
    ([1] * 3, [1000, 24, 37]), ([1] * 5, [2000, 0, 600, 16, 401]), ([1] * 30, [700] * 30),
    ([1] * 37, [600 + 7 * i for i in range(37)]), ([1] * 38, [600 + 7 * i for i in range(38)]),
    ([2, 1], [9000, 400])])
def test_few_short_rows_are_dealt_out(m, ws, fmt, new, total):
    """Calls of so few rows that a CTA gets a part of one, up to as many rows as CTAs."""
    c = Case(390 + len(new), fmt, new, total)
    c.check(c.attend(m, ws, 0, c.sinks), 0, c.sinks)
    c.check(c.attend(m, ws, 391), 391)

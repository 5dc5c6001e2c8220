"""GPU parity of the paged attention against its plain 64-bit value, at the
sizes and masks where it can go wrong.  Tolerances: tests/_paged.py."""
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


def _sinks(c, on):
    return c.sinks if on else None


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("total,window,sinks", [
    ([1], 0, False), ([2], 0, True), ([15], 0, False), ([16], 0, False), ([17], 1, True),
    ([33, 0, 5], 0, True), ([128], 0, False), ([129, 127], 0, False), ([600, 1000, 513], 513, True),
    ([514, 512, 1], 513, False), ([4099], 0, True), ([300] * 40, 0, False), ([70000, 3], 0, True),
    ([20000, 1, 20000], 1000, False)])
def test_next_tokens(m, ws, fmt, total, window, sinks):
    c = Case(11 + len(total) + total[0], fmt, [1] * len(total), total)
    got = c.attend(m, ws, window, _sinks(c, sinks))
    c.check(got, window, _sinks(c, sinks))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total,window,sinks", [
    ([2], [2], 0, False), ([5], [5], 0, True), ([16], [16], 0, False), ([17], [33], 0, False),
    ([4, 1, 3], [1000, 1, 3], 0, True), ([16, 17], [128, 129], 0, False),
    ([100], [100], 7, False), ([100, 30], [700, 1031], 513, True), ([300], [300], 0, True),
    ([129], [4000], 0, False), ([2] * 50, [300] * 50, 100, False), ([515], [1030], 513, False),
    ([3, 0, 2], [12000, 500, 2], 0, False)])
def test_drafts_and_prompts(m, ws, fmt, new, total, window, sinks):
    c = Case(211 + new[0] + total[0], fmt, new, total, page=32)
    got = c.attend(m, ws, window, _sinks(c, sinks))
    c.check(got, window, _sinks(c, sinks))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,nkv", [(8, 8), (1, 1), (2, 1), (4, 2), (8, 4), (16, 4), (64, 8), (4, 1),
                                    (8, 1), (32, 8), (16, 2)])
@pytest.mark.parametrize("new", [1, 37])
def test_head_layouts(m, ws, fmt, nq, nkv, new):
    c = Case(31 + nq + nkv, fmt, [new, 1, new], [200, 77, 40], page=16, nq=nq, nkv=nkv)
    c.check(c.attend(m, ws, 50, c.sinks), 50, c.sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 256, 1024])
@pytest.mark.parametrize("new", [1, 9])
def test_page_sizes(m, ws, fmt, page, new):
    c = Case(41 + page, fmt, [new, new], [page + 3, 3 * page], page=page)
    c.check(c.attend(m, ws))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 20])
def test_rows_behind_the_last_sequence_stay(m, ws, fmt, new):
    c = Case(51, fmt, [new, 0, new], [100, 40, 30], rows_after=13)
    c.check(c.attend(m, ws))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_lengths_shorter_than_the_rows_leave_rows_empty(m, ws, fmt):
    """kv_len below the new rows: the first rows lie before the cache's start."""
    c = Case(52, fmt, [5, 40, 1], [3, 39, 0])
    for sinks in (None, c.sinks):
        got = c.attend(m, ws, sinks=sinks)
        c.check(got, sinks=sinks)
        assert (got[:2] == 0).all() and (got[5] == 0).all() and (got[45] == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_pages_that_are_not_there(m, ws, fmt, new):
    c = Case(53, fmt, [new, new], [400, 300], page=32)
    c.table[0, 2] = c.n_pages          # one past the end
    c.table[0, 5] = -7
    c.table[1, 0] = 0x7FFFFFFF
    c.table[1, 9 if new == 1 else 3] = -1
    keep = c.table.clone()
    c.table = keep.clamp(0, c.n_pages - 1)   # the reference looks rows up, then drops them
    absent = [(0, 2), (0, 5), (1, 0), (1, 9 if new == 1 else 3)]
    b = m.PagedBatch(c.q_start, c.kv_len, keep, c.page, max(c.new))
    got = c.attend(m, ws, batch=b)
    c.check(got, absent=absent)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 24])
def test_evicted_pages_behind_the_window(m, ws, fmt, new):
    """A sliding-window layer keeps no pages behind its window."""
    c = Case(54, fmt, [new], [1000], page=16)
    first = 1000 - new - 100 + 1
    table = c.table.clone()
    table[0, :first // 16] = -1
    b = m.PagedBatch(c.q_start, c.kv_len, table, c.page, new)
    c.check(c.attend(m, ws, 100, batch=b), 100)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 8])
def test_strong_scores_and_uneven_values(m, ws, fmt, new):
    """Scores tens of units apart (a few keys take nearly all weight) and values
    whose loudness differs by orders of magnitude between blocks."""
    c = Case(61, fmt, [new, new], [900, 333], loud=2.0, size=3.0)
    for sinks in (None, 20.0 * c.sinks):
        c.check(c.attend(m, ws, sinks=sinks), sinks=sinks)


def test_block_scales_at_their_limits(m, ws):
    """Blocks whose scales lie at the ends of their range: the loud ones
    dominate, and nothing over- or underflows on the way."""
    for new in (1, 8):
        c = Case(62, "e4m3", [new], [200])
        c.vs[c.rows(0, torch.tensor([0])) // 16] = 2.0 ** 40
        c.vs[c.rows(0, torch.tensor([64])) // 16] = 2.0 ** -40
        c.ks[c.rows(0, torch.tensor([32])) // 16] = 2.0 ** -40
        c.check(c.attend(m, ws))
        c = Case(63, "e4m3", [new], [48])
        c.vs[:] = 2.0 ** -40
        c.check(c.attend(m, ws))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_softmax_scale_and_large_queries(m, ws, fmt):
    for new in (1, 5):
        c = Case(64, fmt, [new], [300])
        for scale in (0.0, 1e-3, 0.5):
            c.check(c.attend(m, ws, scale=scale), scale=scale)
        c.q *= 2.0 ** 60
        c.check(c.attend(m, ws, scale=2.0 ** -63), scale=2.0 ** -63)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total,max_q", [([1, 1, 1], [500, 2, 90], 8), ([1, 4], [4000, 700], 64)])
def test_loose_bound_on_new_tokens(m, ws, fmt, new, total, max_q):
    c = Case(71, fmt, new, total)
    c.check(c.attend(m, ws, max_q=max_q))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3])
def test_many_sequences(m, ws, fmt, new):
    g = torch.Generator().manual_seed(5)
    total = [int(t) for t in torch.randint(new, 200, (256,), generator=g)]
    c = Case(72, fmt, [new] * 256, total)
    c.check(c.attend(m, ws, 60, c.sinks), 60, c.sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total", [([1] * 3, [5000, 17, 9000]), ([70, 1], [3000, 40])])
def test_repeats_and_a_captured_step_give_the_same_bits(m, ws, fmt, new, total):
    c = Case(73, fmt, new, total)
    first = c.attend(m, ws)
    for _ in range(3):
        assert torch.equal(c.attend(m, ws).view(torch.int16), first.view(torch.int16))
    out = torch.full_like(first, 7.25)
    b = c.batch(m)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.attend(m, ws, out=out, batch=b)
    for _ in range(2):
        out.fill_(7.25)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    # The same capture serves other lengths: they are read on the device.
    c.total = [t - 1 for t in c.total]
    c.kv_len.copy_(torch.tensor(c.total, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_two_streams_with_a_workspace_each(m):
    cases = [Case(81, "bf16", [1] * 4, [30000, 20000, 100, 7]), Case(82, "e4m3", [9, 1], [20000, 30000])]
    spaces = [m.new_attn_workspace() for _ in cases]
    alone = [c.attend(m, w) for c, w in zip(cases, spaces)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(5):
        for i, (c, w, st) in enumerate(zip(cases, spaces, streams)):
            with torch.cuda.stream(st):
                outs[i].append(c.attend(m, w, out=torch.full_like(alone[i], 7.25)))
    torch.cuda.synchronize()
    for i, a in enumerate(alone):
        for o in outs[i]:
            assert torch.equal(o.view(torch.int16), a.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 20])
def test_offsets_beyond_31_bits(m, ws, fmt, new):
    """Pages behind the first 2^32 bytes and 2^31 elements of a cache."""
    c = Case(91, fmt, [new], [150], page=64)
    pages = (1 << 31) // (64 * 4 * D) + 40
    if fmt == "e4m3":
        pages = (1 << 32) // (64 * 4 * D) + 40
    table = c.table.clone()
    big = {}
    dims = m.AttnDims(32, 4, D)
    for name in ("k", "v"):
        x = torch.zeros(pages, 64, 4, D, dtype=c.k.dtype, device="cuda")
        src = c.shaped(getattr(c, name))
        for i in range(3):
            x[pages - 1 - i] = src[int(c.table[0, i])]
        big[name] = x
        if fmt == "e4m3":
            s = torch.zeros(pages, 4, 4, device="cuda")
            for i in range(3):
                s[pages - 1 - i] = c.scaled(getattr(c, name + "s"))[int(c.table[0, i])]
            big[name + "s"] = s
    for i in range(3):
        table[0, i] = pages - 1 - i
    b = m.PagedBatch(c.q_start, c.kv_len, table, 64, new)
    out = torch.full_like(c.q, 7.25)
    if fmt == "bf16":
        m.flint_attn_paged_bf16(c.q, big["k"], big["v"], b, out, ws, dims=dims)
    else:
        m.flint_attn_paged_fp8(c.q, big["k"], big["v"], big["ks"], big["vs"], b, out, ws, dims=dims)
    c.check(out)


def test_hostile_batches_stay_in_bounds(m, ws):
    """Row offsets that run backwards or past the rows, lengths below zero or
    past the table: nothing outside the call's rows is written, and the rows a
    sane sequence brings are right."""
    for new in (1, 12):
        c = Case(95, "bf16", [new, new], [100, 60], rows_after=4)
        guard = torch.full((c.T + 64, c.nq, D), 7.25, dtype=torch.bfloat16, device="cuda")
        out = guard[32:32 + c.T]
        for q_start, kv in (([0, new, 1 << 30], [100, 60]), ([-5, new, new + 1], [100, 1 << 30]),
                            ([new, 0, -3], [-9, 60]), ([0, (1 << 31) - 1, 0], [100, 60])):
            b = m.PagedBatch(torch.tensor(q_start, dtype=torch.int32, device="cuda"),
                             torch.tensor(kv, dtype=torch.int32, device="cuda"), c.table, c.page, new)
            c.attend(m, ws, out=out, batch=b)
        torch.cuda.synchronize()
        assert (guard[:32] == 7.25).all() and (guard[32 + c.T:] == 7.25).all()
        out.fill_(7.25)
        c.check(c.attend(m, ws, out=out))

"""flint_linear_bf16 and flint_grouped_linear_bf16 against 64 bits: sizes around every tile
border, activations, bias, residual, types; ragged, empty and clamped groups."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p

pytestmark = pytest.mark.gpu
ACTS = [p.NONE, p.SILU, p.GELU, p.SWIGLU]


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


def _case(rows, n_in, n_out, act, bias, residual, dtype, seed=0):
    g = p.gen(seed + rows + 7 * n_in + 13 * n_out)
    mr = n_out * (2 if act == p.SWIGLU else 1)
    x, w = p.bf(g, rows, n_in), p.bf(g, mr, n_in, scale=n_in ** -0.5)
    b = torch.randn(mr, generator=g, device="cuda") if bias else None
    r = torch.randn(rows, n_out, generator=g, device="cuda").to(dtype) if residual else None
    return x, w, b, r


def _run(ws, x, w, b, r, act, dtype, n_out):
    """The call, into the middle of a larger buffer whose ends have to stay."""
    rows = x.shape[0]
    big = torch.full((rows + 2, n_out), 7.0, device="cuda", dtype=dtype)
    m.flint_linear_bf16(x, w, big[1:-1], ws, bias=b, residual=r, act=act)
    assert (big[0] == 7).all() and (big[-1] == 7).all()
    return big[1:-1]


ROWS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 511,
        513, 1021, 2050]


@pytest.mark.parametrize("rows", ROWS)
def test_rows(ws, rows):
    for n_in, n_out, act, dtype in ((520, 264, p.NONE, torch.bfloat16), (256, 400, p.SWIGLU, torch.bfloat16)):
        x, w, b, r = _case(rows, n_in, n_out, act, True, True, dtype)
        p.check(_run(ws, x, w, b, r, act, dtype, n_out), p.linear(x, w, b, r, act, dtype), (n_in, n_out))


@pytest.mark.parametrize("n_in", [8, 16, 24, 56, 64, 72, 120, 128, 136, 504, 1032, 4096, 8200])
@pytest.mark.parametrize("rows", [3, 40, 333])
def test_inputs(ws, n_in, rows):
    for act in (p.NONE, p.SWIGLU):
        x, w, b, r = _case(rows, n_in, 48, act, False, False, torch.bfloat16)
        p.check(_run(ws, x, w, b, r, act, torch.bfloat16, 48), p.linear(x, w, b, r, act, torch.bfloat16))


@pytest.mark.parametrize("n_out", [8, 16, 24, 40, 48, 56, 64, 72, 120, 128, 136, 248, 256, 272, 504, 1000, 2048,
                                   5120])
@pytest.mark.parametrize("rows", [1, 50, 290])
def test_outputs(ws, n_out, rows):
    for act in (p.NONE, p.SWIGLU):
        if act == p.SWIGLU and n_out % 16:
            continue
        for dtype in (torch.bfloat16, torch.float32):
            x, w, b, r = _case(rows, 192, n_out, act, True, True, dtype)
            p.check(_run(ws, x, w, b, r, act, dtype, n_out), p.linear(x, w, b, r, act, dtype), (act, dtype))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [5, 30, 70, 600])
def test_epilogues(ws, act, dtype, rows):
    for bias in (False, True):
        for residual in (False, True):
            x, w, b, r = _case(rows, 200, 144, act, bias, residual, dtype)
            p.check(_run(ws, x, w, b, r, act, dtype, 144), p.linear(x, w, b, r, act, dtype), (bias, residual))


@pytest.mark.parametrize("rows", [4, 44, 444])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_residual_in_place(ws, rows, dtype):
    x, w, b, r = _case(rows, 136, 520, p.NONE, True, True, dtype)
    want = p.linear(x, w, b, r, p.NONE, dtype)
    m.flint_linear_bf16(x, w, r, ws, bias=b, residual=r)
    p.check(r, want)


@pytest.mark.parametrize("rows", [6, 60, 700])
def test_large_and_special_values(ws, rows):
    """Activations at the ends of their range; an infinity or NaN stays with its row, and a
    NaN weight with its output."""
    g = p.gen(rows)
    x, w = p.bf(g, rows, 64), p.bf(g, 64, 64, scale=40.0)   # sums of hundreds
    for act in (p.SILU, p.GELU):
        p.check(_run(ws, x, w, None, None, act, torch.bfloat16, 64), p.linear(x, w, None, None, act, torch.bfloat16))
    want = _run(ws, x, w, None, None, p.NONE, torch.bfloat16, 64).clone()
    x[rows // 2, 3], x[rows - 1, 63] = float("nan"), float("inf")
    w[17, 5] = float("nan")
    got = _run(ws, x, w, None, None, p.NONE, torch.bfloat16, 64)
    bad = torch.zeros(rows, 64, dtype=torch.bool, device="cuda")
    bad[rows // 2], bad[rows - 1], bad[:, 17] = True, True, True
    assert torch.equal(got[~bad], want[~bad])
    assert not torch.isfinite(got[bad]).any()


def test_same_bits_again(ws):
    for rows in (3, 33, 1500):
        x, w, b, r = _case(rows, 2048, 1024, p.NONE, True, True, torch.bfloat16)
        first = _run(ws, x, w, b, r, p.NONE, torch.bfloat16, 1024).clone()
        for _ in range(3):
            assert torch.equal(first, _run(ws, x, w, b, r, p.NONE, torch.bfloat16, 1024))


@pytest.mark.parametrize("rows", [2, 48, 520])
def test_streams_and_graphs(ws, rows):
    """On a stream that is not the default one, and captured: replays read the inputs anew."""
    x, w, b, r = _case(rows, 512, 256, p.SWIGLU, True, False, torch.bfloat16)
    out = torch.empty(rows, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.flint_linear_bf16(x, w, out, ws, bias=b, act=p.SWIGLU)
    torch.cuda.current_stream().wait_stream(s)
    p.check(out, p.linear(x, w, b, r, p.SWIGLU, torch.bfloat16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.flint_linear_bf16(x, w, out, ws, bias=b, act=p.SWIGLU)
    for seed in (1, 2):
        x.copy_(p.bf(p.gen(seed), rows, 512))
        out.zero_()
        graph.replay()
        p.check(out, p.linear(x, w, b, r, p.SWIGLU, torch.bfloat16))


def test_weights_written_just_before(ws):
    """The call reads weights, rows and bias that the kernel before it wrote."""
    for rows in (1, 40, 700):
        x, w, b, _ = _case(rows, 1024, 2048, p.NONE, True, False, torch.bfloat16)
        w2, x2, b2 = torch.empty_like(w), torch.empty_like(x), torch.empty_like(b)
        out = torch.empty(rows, 2048, dtype=torch.bfloat16, device="cuda")
        for i in range(4):
            w2.copy_(w), x2.copy_(x), b2.copy_(b)
            torch.mul(w, 1 if i % 2 else -1, out=w2)
            m.flint_linear_bf16(x2, w2, out, ws, bias=b2)
            want = p.linear(x2, w2, b2, None, p.NONE, torch.bfloat16)
            p.check(out, want, (rows, i))


def _check_groups(ws, sizes, n_in, n_out, act, n_x=None, bias=False, dtype=torch.bfloat16, seed=1,
                  start=None, rows=None, index=None):
    g = p.gen(seed)
    mr = n_out * (2 if act == p.SWIGLU else 1)
    if start is None:
        start = [0]
        for n in sizes:
            start.append(start[-1] + n)
    groups, rows = len(start) - 1, start[-1] if rows is None else rows
    if n_x is not None and index is None:
        index = torch.randint(0, n_x, (rows,), generator=g, device="cuda", dtype=torch.int32)
    x = p.bf(g, rows if n_x is None else n_x, n_in)
    w = p.bf(g, groups, mr, n_in, scale=n_in ** -0.5)
    b = torch.randn(groups, mr, generator=g, device="cuda") if bias else None
    out = torch.full((rows, n_out), 7.0, device="cuda", dtype=dtype)
    starts = torch.tensor(start, dtype=torch.int32, device="cuda")
    m.flint_grouped_linear_bf16(x, w, starts, out, ws, row_index=index, bias=b, act=act)
    want = p.grouped(x, w, start, None if index is None else index.tolist(), b, act, dtype, rows)
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    if want:
        at = torch.tensor(sorted(want), device="cuda")
        hit[at] = True
        p.check(out[at], (torch.stack([want[i][0] for i in at.tolist()]),
                          torch.stack([want[i][1] for i in at.tolist()])))
    assert (out[~hit] == 7).all()


GROUPS = [[1], [0, 1, 0], [5, 0, 3], [0, 0, 300, 1, 0], [32, 33, 31, 64, 65], [255, 256, 257],
          [1] * 40, [3, 700, 2, 0, 129], [513, 0, 0, 40]]


@pytest.mark.parametrize("sizes", GROUPS)
@pytest.mark.parametrize("act", [p.NONE, p.SWIGLU])
def test_groups(ws, sizes, act):
    _check_groups(ws, sizes, 200, 144, act, bias=True)
    _check_groups(ws, sizes, 128, 272, act, n_x=max(1, sum(sizes) // 3))


@pytest.mark.parametrize("act", [p.SILU, p.GELU])
def test_groups_other_epilogues(ws, act):
    _check_groups(ws, [3, 0, 90, 300], 72, 40, act, bias=True, dtype=torch.float32)
    _check_groups(ws, [3, 0, 90, 300], 72, 40, act, bias=True, n_x=50)


def test_many_groups(ws):
    g = torch.Generator().manual_seed(5)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    _check_groups(ws, sizes, 64, 32, p.NONE, n_x=77)
    _check_groups(ws, [0] * 1023 + [9], 64, 32, p.SWIGLU)
    _check_groups(ws, [9] + [0] * 1023, 64, 32, p.SWIGLU)


def test_expert_shapes(ws):
    """The layer's own products, ragged as a short prompt routes them."""
    g = torch.Generator().manual_seed(6)
    sizes = torch.randint(0, 12, (64,), generator=g).tolist()
    _check_groups(ws, sizes, 2048, 512, p.SWIGLU, n_x=100)
    _check_groups(ws, sizes, 512, 2048, p.NONE)


def test_rows_of_no_group_and_bad_indices(ws):
    for scale in (1, 20):
        at = [4, 10, 10, 17]
        _check_groups(ws, None, 64, 48, p.NONE, start=[scale * a for a in at], rows=20 * scale)
        idx = torch.arange(20 * scale, dtype=torch.int32, device="cuda") % 9
        idx[::3] = -1
        idx[1::5] = 9
        idx[7] = 2 ** 31 - 1
        _check_groups(ws, None, 64, 48, p.SWIGLU, start=[scale * a for a in at], rows=20 * scale, n_x=9, index=idx)


def test_starts_out_of_range_are_clamped(ws):
    _check_groups(ws, None, 64, 48, p.NONE, start=[-5, 3, 8, 2 ** 31 - 1], rows=40)
    _check_groups(ws, None, 64, 48, p.NONE, start=[2 ** 31 - 1, 50, 60, 90], rows=40)
    _check_groups(ws, None, 64, 48, p.NONE, start=[-2 ** 31, -7, 0, 0], rows=40)
    _check_groups(ws, None, 64, 48, p.NONE, start=[30, 20, 25, 25], rows=40)   # the first ends early


@pytest.mark.parametrize("act", ACTS)
def test_few_rows_in_groups(ws, act):
    """Up to nine rows in all (both sides of a kernel's limit): any number of groups, gathered,
    bad indices, rows of no group, hostile starts, long rows."""
    for dtype in (torch.bfloat16, torch.float32):
        for sizes in ([1], [8], [9], [3, 0, 5], [0, 0, 1, 0, 7], [1] * 8, [0] * 700 + [4] + [0] * 323):
            _check_groups(ws, sizes, 72, 48, act, bias=True, dtype=dtype)
            _check_groups(ws, sizes, 72, 48, act, n_x=3, dtype=dtype)
    _check_groups(ws, [2, 0, 6], 4104, 144, act, bias=True)
    idx = torch.tensor([0, -1, 5, 2, 2 ** 31 - 1, 4, 4], dtype=torch.int32, device="cuda")
    _check_groups(ws, None, 64, 48, act, start=[1, 3, 3, 6], rows=7, n_x=5, index=idx)
    for start in ([-5, 3, 8, 2 ** 31 - 1], [2 ** 31 - 1, 5, 6, 9], [-2 ** 31, -7, 0, 0], [6, 2, 4, 4], [0, 0, 0, 0]):
        _check_groups(ws, None, 64, 48, act, start=start, rows=7)


def test_empty_groups_weights_do_not_matter(ws):
    g = p.gen(3)
    x, w = p.bf(g, 12, 64), p.bf(g, 3, 32, 64, scale=0.125)
    start = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device="cuda")
    out, out2 = (torch.zeros(12, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.flint_grouped_linear_bf16(x, w, start, out, ws)
    w[1] = float("nan")
    m.flint_grouped_linear_bf16(x, w, start, out2, ws)
    assert torch.equal(out, out2)


def test_group_neighbours_do_not_leak(ws):
    """NaN rows of one group never reach another one's, inside a tile or not."""
    g = p.gen(4)
    x, w = p.bf(g, 300, 64), p.bf(g, 3, 32, 64, scale=0.125)
    x[100:110] = float("nan")
    start = torch.tensor([0, 100, 110, 300], dtype=torch.int32, device="cuda")
    out = torch.zeros(300, 32, dtype=torch.bfloat16, device="cuda")
    m.flint_grouped_linear_bf16(x, w, start, out, ws)
    assert torch.isfinite(out[:100]).all() and torch.isfinite(out[110:]).all()
    assert torch.isnan(out[100:110]).all()


def test_binding_refuses(ws):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    ok = dict(x=x, w=w, out=out, workspace=ws)
    m.flint_linear_bf16(**ok)
    for bad in (dict(x=x.float()), dict(x=x[:, ::2]), dict(w=w.T), dict(w=w[:, :56]), dict(out=out.half()),
                dict(out=out[:3]), dict(bias=torch.zeros(31, device="cuda")), dict(bias=out[0]),
                dict(residual=out.float()), dict(residual=out[:2]), dict(act=4), dict(act=1.0),
                dict(act=p.SWIGLU), dict(workspace=ws[:64]), dict(workspace=ws.view(torch.int8)),
                dict(w=w.cpu()), dict(x=x.cpu()), dict(out=x[:, :32])):
        with pytest.raises(m.FlintError):
            m.flint_linear_bf16(**{**ok, **bad})
    start = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ok = dict(x=x, w=w[None], group_start=start, out=out, workspace=ws)
    m.flint_grouped_linear_bf16(**ok)
    for bad in (dict(group_start=start.long()), dict(group_start=start[:1]), dict(x=x[:3]),
                dict(row_index=start), dict(row_index=torch.zeros(4, device="cuda")), dict(w=w),
                dict(bias=torch.zeros(32, device="cuda"))):
        with pytest.raises(m.FlintError):
            m.flint_grouped_linear_bf16(**{**ok, **bad})

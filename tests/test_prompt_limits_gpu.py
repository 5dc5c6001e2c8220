"""The linear side of a prompt at its limits: the largest sizes, tensors of more than 2^31
elements, many groups, every token on the same experts, two streams at once, NaN tokens."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p
from tests.test_moe_prompt_gpu import _check_layer, _layer_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def layer():
    return fs.layer_weights(1001, fs.FULL, device="cuda")


def _some(n, k=200):
    """A few of n rows: the first, the last, some between."""
    g = torch.Generator().manual_seed(n)
    return torch.cat([torch.arange(min(n, 3)), torch.arange(max(0, n - 3), n),
                      torch.randint(0, n, (k,), generator=g)]).unique().cuda()


@pytest.mark.parametrize("rows,n_in,n_out,act", [
    (65536, 64, 64, p.NONE), (65536, 16, 48, p.SWIGLU), (1, 65536, 64, p.NONE), (7, 65536, 32, p.SWIGLU),
    (50, 65536, 40, p.NONE), (1, 16, 1 << 20, p.NONE), (3, 8, 1 << 20, p.SWIGLU), (40, 24, 1 << 20, p.NONE),
    (300, 40, 1 << 19, p.SWIGLU)])
def test_largest_sizes(ws, rows, n_in, n_out, act):
    g = p.gen(rows + n_in)
    x, w = p.bf(g, rows, n_in), p.bf(g, n_out * (2 if act == p.SWIGLU else 1), n_in, scale=n_in ** -0.5)
    out = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda")
    m.flint_linear_bf16(x, w, out, ws, act=act)
    r, f = _some(rows), _some(n_out)
    wf = w[torch.cat([f, f + n_out])] if act == p.SWIGLU else w[f]
    p.check(out[r][:, f], p.linear(x[r], wf, None, None, act, torch.bfloat16))


@pytest.mark.parametrize("what", ["out", "w", "x"])
def test_more_than_2_31_elements(ws, what):
    rows, n_in, n_out = {"out": (65536, 64, 40000), "w": (20, 2104, 1 << 20), "x": (65536, 32784, 64)}[what]
    assert {"out": rows * n_out, "w": n_in * n_out, "x": rows * n_in}[what] > 2 ** 31
    g = p.gen(1)
    x, w = p.bf(g, rows, n_in), p.bf(g, n_out, n_in, scale=n_in ** -0.5)
    out = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda")
    m.flint_linear_bf16(x, w, out, ws)
    r, f = _some(rows), _some(n_out)
    p.check(out[r][:, f], p.linear(x[r], w[f], None, None, p.NONE, torch.bfloat16))


def test_groups_of_more_than_2_31_weights(ws):
    """Weights of 1024 groups, rows in the last ones: offsets beyond 32 bits."""
    g = p.gen(2)
    groups, n_in, n_out = 1024, 1024, 2056
    w = torch.empty(groups, n_out, n_in, dtype=torch.bfloat16, device="cuda")
    for i in range(0, groups, 64):
        w[i:i + 64] = p.bf(g, 64, n_out, n_in, scale=n_in ** -0.5)
    assert w.numel() > 2 ** 31
    sizes = [0] * groups
    sizes[0], sizes[1021], sizes[1023] = 5, 300, 40
    start = [0]
    for n in sizes:
        start.append(start[-1] + n)
    x = p.bf(g, start[-1], n_in)
    out = torch.empty(start[-1], n_out, dtype=torch.bfloat16, device="cuda")
    m.flint_grouped_linear_bf16(x, w, torch.tensor(start, dtype=torch.int32, device="cuda"), out, ws)
    for i in (0, 1021, 1023):
        a, b = start[i], start[i + 1]
        p.check(out[a:b], p.linear(x[a:b], w[i], None, None, p.NONE, torch.bfloat16), i)


def test_65536_rows_of_one_token(ws):
    """Every row of the largest call the same row of x, in a few groups."""
    g = p.gen(3)
    x, w = p.bf(g, 1, 72), p.bf(g, 3, 64, 72, scale=72 ** -0.5)
    start = torch.tensor([0, 1, 65000, 65536], dtype=torch.int32, device="cuda")
    index = torch.zeros(65536, dtype=torch.int32, device="cuda")
    out = torch.empty(65536, 64, dtype=torch.bfloat16, device="cuda")
    m.flint_grouped_linear_bf16(x, w, start, out, ws, row_index=index)
    for i, (a, b) in enumerate([(0, 1), (1, 65000), (65000, 65536)]):
        y, e = p.linear(x, w[i], None, None, p.NONE, torch.bfloat16)
        p.check(out[a:b], (y.expand(b - a, -1), e.expand(b - a, -1)), i)


def test_layer_of_8192_tokens(layer):
    x, res = fs.tokens(77, 8192, device="cuda")
    offset = fs.logit_offsets(1003, device="cuda")
    ws, out = m.new_prompt_workspace(8192), torch.empty_like(res)
    args = (layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"], layer["ws2"])
    m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    _check_layer(out, _layer_ref(x, res, layer, offset, False))
    again = torch.empty_like(out)
    m.flint_moe_prompt_bf16(x, res, *args, again, ws)
    assert torch.equal(out, again)


def test_layer_on_six_experts(layer):
    """Every token on the same six experts (offsets of 60 logits, that only choose)."""
    x, res = fs.tokens(78, 1300, device="cuda")
    offset = torch.zeros(256, device="cuda")
    offset[[0, 17, 100, 101, 254, 255]] = torch.arange(60.0, 360.0, 50.0, device="cuda")
    ws, out = m.new_prompt_workspace(1300), torch.empty_like(res)
    idx = torch.empty(1300, 6, dtype=torch.int32, device="cuda")
    m.flint_moe_prompt_bf16(x, res, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, ws, idx, dims=m.SELECT_DIMS)
    assert (idx == torch.tensor([255, 254, 101, 100, 17, 0], device="cuda")).all()
    _check_layer(out, _layer_ref(x, res, layer, offset, True))


def test_layer_with_a_nan_token(layer):
    """A token of NaN is NaN, and nobody else is."""
    x, res = fs.tokens(79, 200, device="cuda")
    args = (layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"], layer["ws2"])
    ws, out, want = m.new_prompt_workspace(200), torch.empty_like(res), torch.empty_like(res)
    x[57] = 0
    m.flint_moe_prompt_bf16(x, res, *args, want, ws)
    x[57] = float("nan")
    m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    others = torch.arange(200, device="cuda") != 57
    # (the token's zeros chose other experts than its NaN: rows move, sums do not)
    assert torch.equal(out[others], want[others])
    assert torch.isnan(out[57]).all()


def test_two_streams_at_once(ws):
    """Tiled kernels of two streams, each with its workspace, and a selection beside them."""
    g = p.gen(5)
    a, b = (p.bf(g, 700, 1024) for _ in range(2))
    w = p.bf(g, 2048, 1024, scale=1024 ** -0.5)
    logits = torch.randn(900, 256, generator=g, device="cuda")
    other, s = m.new_prompt_workspace(), torch.cuda.Stream()
    outs = [torch.empty(700, 2048, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    sel = (i32(900, 6), torch.empty(900, 6, device="cuda"), i32(257), i32(5400), i32(900, 6))
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        m.flint_linear_bf16(a, w, outs[0], ws)
        with torch.cuda.stream(s):
            m.flint_linear_bf16(b, w, outs[1], other)
            m.flint_moe_select(logits, None, *sel, other)
    torch.cuda.current_stream().wait_stream(s)
    p.check(outs[0], p.linear(a, w, None, None, p.NONE, torch.bfloat16))
    p.check(outs[1], p.linear(b, w, None, None, p.NONE, torch.bfloat16))
    assert torch.equal(sel[0].long(), p.choose(logits, None, False)[0])
    assert m.flint_prompt_get_device_status(other) == m.FLINT_OK

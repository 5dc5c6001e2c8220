"""flint_moe_select, flint_moe_combine_bf16 and flint_moe_prompt_bf16 against 64 bits, and a
decoder layer's calls in a row."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p
from tests._util import TAU

pytestmark = pytest.mark.gpu
E, K, H = 256, 6, 2048


@pytest.fixture(scope="module")
def ws():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    w = m.new_prompt_workspace()
    yield w
    torch.cuda.synchronize()
    assert m.flint_prompt_get_device_status(w) == m.FLINT_OK


@pytest.fixture(scope="module")
def layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return fs.layer_weights(1001, fs.FULL, device="cuda")


def _select(ws, logits, offset=None, dims=None):
    n = logits.shape[0]
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = (i32(n, K), torch.full((n, K), -9.0, device="cuda"), i32(E + 1), i32(n * K), i32(n, K))
    m.flint_moe_select(logits, offset, *out, ws, dims=dims)
    return out


def _check_select(ws, logits, offset=None, dims=None):
    idx, w, start, row_token, pair_row = _select(ws, logits, offset, dims)
    want, weight = p.choose(logits, offset, dims is m.SELECT_DIMS)
    assert torch.equal(idx.long(), want)
    finite = torch.isfinite(weight)
    assert torch.equal(finite, torch.isfinite(w))
    # a sigmoid: exp within 2 units of the last place, an addition, a division; a sum of six, a
    # division: 16 half steps of fp32 in all
    off = (w.double() - weight).abs() - (16 * 2.0 ** -24 * weight + 1e-38)
    assert (off[finite] <= 0).all(), float(off[finite].max())
    s, t, r = p.order_of(idx)
    assert torch.equal(start.long(), s) and torch.equal(row_token.long(), t)
    assert torch.equal(pair_row.long(), r)


@pytest.mark.parametrize("n", [1, 2, 8, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 1000, 4097, 8191, 8192])
def test_select_sizes(ws, n):
    g = p.gen(n)
    logits = torch.randn(n, E, generator=g, device="cuda")
    offset = torch.randn(E, generator=g, device="cuda")
    _check_select(ws, logits)
    _check_select(ws, logits, offset)
    _check_select(ws, logits, offset, m.SELECT_DIMS)


def test_select_ties(ws):
    """Scores of few values, equal ones all, zeros of both signs, one expert for everybody."""
    g = p.gen(1)
    for n in (5, 300):
        _check_select(ws, torch.randint(-2, 3, (n, E), generator=g, device="cuda").float())
        _check_select(ws, torch.zeros(n, E, device="cuda"))
        z = torch.zeros(n, E, device="cuda")
        z[:, ::3] = -0.0
        _check_select(ws, z)
        one = torch.randn(n, E, generator=g, device="cuda")
        one[:, 250:] += 100.0
        _check_select(ws, one)


def test_select_masks(ws):
    """Experts masked by the lowest value or -infinity, all but one, and all of them."""
    g = p.gen(2)
    for n in (3, 130):
        logits = torch.randn(n, E, generator=g, device="cuda")
        for low in (torch.finfo(torch.float32).min, float("-inf")):
            off = torch.zeros(E, device="cuda")
            off[8:] = low
            _check_select(ws, logits, off)
            _check_select(ws, logits, off, m.SELECT_DIMS)
            off[:] = low
            off[77] = 0
            _check_select(ws, logits, off)
            off[77] = low
            _check_select(ws, logits, off)
            idx, w, *_ = _select(ws, logits, off)
            assert (w == 0).all()


def test_select_infinities_and_nan(ws):
    g = p.gen(3)
    logits = torch.randn(70, E, generator=g, device="cuda")
    logits[3, 200] = logits[3, 9] = float("inf")
    logits[4, 200] = float("nan")
    logits[5, 100] = torch.tensor(-1, dtype=torch.int32).view(torch.float32)   # a NaN with its sign
    logits[6, 10:] = float("-inf")
    logits[7, 0], logits[7, 1] = float("nan"), float("inf")
    logits[69] = float("nan")
    _check_select(ws, logits)


def test_select_in_a_graph(ws):
    logits = torch.randn(500, E, generator=p.gen(4), device="cuda")
    out = _select(ws, logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.flint_moe_select(logits, None, *out, ws)
    logits.copy_(torch.randn(500, E, generator=p.gen(5), device="cuda"))
    graph.replay()
    for a, b in zip(out, _select(ws, logits)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 3, 100, 2000])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_combine(n, shared, in_place):
    g = p.gen(n)
    res, y = p.bf(g, n, H), p.bf(g, n * K, H)
    ys = p.bf(g, n, H) if shared else None
    w = torch.rand(n, K, generator=g, device="cuda")
    row = torch.randperm(n * K, generator=g, device="cuda").to(torch.int32).view(n, K)
    if n > 2:
        row[1, 2], row[2, 5], row[2, 0] = -1, n * K, 2 ** 31 - 1   # add nothing
        w[1, 2] = float("nan")
    ok = (row >= 0) & (row < n * K)
    terms = torch.where(ok[..., None], w.double()[..., None] * y[torch.where(ok, row, 0).long()].double(), 0)
    want = res.double() + terms.sum(1) + (ys.double() if shared else 0)
    size = res.double().abs() + terms.abs().sum(1) + (ys.double().abs() if shared else 0)
    out = res if in_place else torch.empty_like(res)
    m.flint_moe_combine_bf16(res, y, row, w, ys, out)
    err = 8 * 2.0 ** -24 * size   # eight roundings of sums no larger
    p.check(out, (want, err + 2.0 ** -8 * (want.abs() + err) + 1e-38))


W_TOL = 1e-5    # of a routing weight: checked of its own, and a part of the outputs' bound
HALF = 2.0 ** -8   # half a step of bf16, relative


def _layer_ref(x, res, W, offset, select_only):
    """(out, how far each output may be off, what the experts' terms' squares sum to,
    experts, weights, gaps between the 7 best scores) in 64 bits.

    An output is res + y_s + sum_j w_j y_j, y = bf16(w2 bf16(h)): an h is off by what
    p.linear() says of a bf16 output, which reaches y times |w2|; y has 512 fp32 additions
    and its own half step; the sum 8 fp32 additions and the output's half step."""
    X = x.double()
    score = X @ W["wr"].double().T
    key = score if offset is None else score + offset.double()
    top = key.topk(K + 1, dim=1)
    idx = top.indices[:, :K]
    s = torch.sigmoid((score if select_only else key).gather(1, idx))
    w = s / s.sum(1, keepdim=True)

    def ffn(v, w13, w2):
        h, eh = p.linear(v, w13, None, None, p.SWIGLU, torch.bfloat16)
        w2 = w2.double().T
        y = h @ w2
        e = eh @ w2.abs() + 528 * p.ADD * ((h.abs() + eh) @ w2.abs())
        return y, e + HALF * (y.abs() + e)

    y, err = ffn(x, W["ws13"][0], W["ws2"][0])
    out, square = res.double() + y, y ** 2
    size = res.double().abs() + y.abs()
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        y, ey = ffn(x[t], W["w13"][e], W["w2"][e])
        wy = w[t, j, None] * y
        out.index_add_(0, t, wy)
        err.index_add_(0, t, (w[t, j, None] + W_TOL) * ey + W_TOL * y.abs())
        square.index_add_(0, t, wy ** 2)
        size.index_add_(0, t, wy.abs())
    err = err + 8 * 2.0 ** -24 * size
    return out, err + HALF * (out.abs() + err), square, idx, w, top.values[:, :-1] - top.values[:, 1:]


def _check_layer(out, ref):
    """Outputs of the tokens whose experts are settled: each within its bound; and, as the
    errors of h, of y and of the output are roundings of one sign as often as the other, all
    together within half steps whose squares add: the output's, and of every term two."""
    want, err, square, _, _, gaps = ref
    sure = gaps[:, K - 1] >= TAU
    assert int(sure.sum()) >= 0.9 * len(sure)
    p.check(out[sure], (want[sure], err[sure]))
    norm = float((out[sure].double() - want[sure]).square().sum().sqrt())
    assert norm <= HALF * float((want[sure].square() + 2 * square[sure]).sum().sqrt())
    return sure


@pytest.mark.parametrize("n", [1, 2, 9, 40, 128, 129, 150, 257, 700, 1500])
@pytest.mark.parametrize("mode", ["none", "logit", "select"])
def test_layer(layer, n, mode):
    x, res = fs.tokens(2000 + n, n, device="cuda")
    offset = None if mode == "none" else fs.logit_offsets(1003, device="cuda")
    dims = m.SELECT_DIMS if mode == "select" else m.FULL_DIMS
    ws = m.new_prompt_workspace(n)
    out = torch.empty_like(res)
    idx = torch.full((n, K), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(n, K, device="cuda")
    m.flint_moe_prompt_bf16(x, res, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, ws, idx, w, dims=dims)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    ref = _layer_ref(x, res, layer, offset, mode == "select")
    _, _, _, ref_idx, ref_w, gaps = ref
    sure = _check_layer(out, ref)
    ranked = sure & (gaps.amin(1) >= TAU)  # the experts' order is settled too
    assert torch.equal(idx[ranked].long(), ref_idx[ranked])
    assert torch.equal(idx[sure].sort(1).values.long(), ref_idx[sure].sort(1).values)
    assert int(ranked.sum()) >= 0.8 * n
    assert float((w[ranked].double() - ref_w[ranked]).abs().max()) <= W_TOL
    # in place, without the optional outputs: the same bits
    again = res.clone()
    m.flint_moe_prompt_bf16(x, again, layer["wr"], offset, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], again, ws, dims=dims)
    assert torch.equal(again, out)


def test_layer_is_its_parts(layer):
    """The public calls in a row give the layer's bits, and a larger workspace too."""
    n = 333
    x, res = fs.tokens(5, n, device="cuda")
    ws, big = m.new_prompt_workspace(n), m.new_prompt_workspace(2 * n)
    outs = []
    for w in (ws, big):
        outs.append(torch.empty_like(res))
        m.flint_moe_prompt_bf16(x, res, layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"],
                                layer["ws2"], outs[-1], w)
    assert torch.equal(*outs)
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    logits = torch.empty(n, E, device="cuda")
    m.flint_linear_bf16(x, layer["wr"], logits, ws)
    idx, wt, start, row_token, pair_row = _select(ws, logits)
    h, y, hs, ys, out = bf(n * K, 512), bf(n * K, H), bf(n, 512), bf(n, H), bf(n, H)
    m.flint_grouped_linear_bf16(x, layer["w13"], start, h, ws, row_index=row_token, act=p.SWIGLU)
    m.flint_grouped_linear_bf16(h, layer["w2"], start, y, ws)
    m.flint_linear_bf16(x, layer["ws13"][0], hs, ws, act=p.SWIGLU)
    m.flint_linear_bf16(hs, layer["ws2"][0], ys, ws)
    m.flint_moe_combine_bf16(res, y, pair_row, wt, ys, out)
    ref = _layer_ref(x, res, layer, None, False)
    _check_layer(out, ref)
    _check_layer(outs[0], ref)


@pytest.mark.parametrize("n", [3, 64, 128])
def test_layer_is_the_decode_call_for_few_tokens(layer, n):
    """Bit for bit, in a workspace of its own and in one that larger calls use in between."""
    x, res = fs.tokens(6, n, device="cuda")
    args = (layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"], layer["ws2"])
    want = torch.empty_like(res)
    m.flint_moe_decode_bf16(x, res, *args, want, m.new_workspace(n))
    more, more_res = fs.tokens(7, 300, device="cuda")
    big = m.new_prompt_workspace(300)
    for ws in (m.new_prompt_workspace(n), big, big):
        out = torch.empty_like(res)
        m.flint_moe_prompt_bf16(x, res, *args, out, ws)
        assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
        assert torch.equal(out, want)
        if ws is big:
            m.flint_moe_prompt_bf16(more, more_res, *args, torch.empty_like(more), big)
            assert m.flint_prompt_get_device_status(big) == m.FLINT_OK


def test_layer_against_the_decode_call(layer):
    """The decode call, whose intermediates are exact to 2^-16, is within the same bounds."""
    n = 200
    x, res = fs.tokens(6, n, device="cuda")
    out, dec = torch.empty_like(res), torch.empty_like(res)
    m.flint_moe_decode_bf16(x, res, layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], dec, m.new_workspace(n))
    m.flint_moe_prompt_bf16(x, res, layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"],
                            layer["ws2"], out, m.new_prompt_workspace(n))
    ref = _layer_ref(x, res, layer, None, False)
    _check_layer(out, ref)
    _check_layer(dec, ref)


@pytest.mark.parametrize("n", [5, 40, 300])
def test_layer_in_a_graph(layer, n):
    x, res = fs.tokens(7, n, device="cuda")
    ws, out = m.new_prompt_workspace(n), torch.empty_like(res)
    args = (layer["wr"], None, layer["w13"], layer["w2"], layer["ws13"], layer["ws2"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.flint_moe_prompt_bf16(x, res, *args, out, ws)
    for seed in (8, 9):
        nx, nr = fs.tokens(seed, n, device="cuda")
        x.copy_(nx), res.copy_(nr)
        graph.replay()
        want = torch.empty_like(out)
        m.flint_moe_prompt_bf16(nx, nr, *args, want, m.new_prompt_workspace(n))
        assert torch.equal(out, want)


@pytest.mark.parametrize("n", [257, 1000, 8192])
def test_rmsnorm_of_a_prompt(n):
    """The norm in front of the experts for more rows than a decode step has: the bits of
    calls of 256 rows each, which are within two roundings of 64 bits."""
    x, _ = fs.tokens(12, n, device="cuda")
    x = (x.float() * torch.linspace(0.01, 30, n, device="cuda")[:, None]).bfloat16()
    out, parts = torch.empty_like(x), torch.empty_like(x)
    m.flint_moe_rmsnorm_bf16(x, out)
    for i in range(0, n, 256):
        m.flint_moe_rmsnorm_bf16(x[i:i + 256], parts[i:i + 256])
    assert torch.equal(out, parts)
    d = x.double()
    want = d / (d.square().mean(1, keepdim=True) + 1e-6).sqrt()
    p.check(out, (want, HALF * want.abs() + 2.0 ** -18 * want.abs() + 1e-38))
    with pytest.raises(m.FlintError):
        m.flint_moe_rmsnorm_bf16(torch.zeros(8193, H, dtype=torch.bfloat16, device="cuda"),
                                 torch.zeros(8193, H, dtype=torch.bfloat16, device="cuda"))


def test_a_decoder_layer(layer):
    """Projection, append, attention, output projection into the residual stream, and the
    experts: two prompts through one layer, against 64 bits step by step."""
    lens, page = [137, 75], 16
    n = sum(lens)
    g = p.gen(11)
    x, res = fs.tokens(10, n, device="cuda")
    w_qkv, w_o = p.bf(g, 40 * 128, H, scale=H ** -0.5), p.bf(g, H, 32 * 128, scale=4096 ** -0.5)
    gain = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32(*(list(range(9)) + [9, 10, 11, 12, 13, -1, -1, -1, -1])).view(2, 9)
    batch = m.PagedBatch(i32(0, lens[0], n), i32(*lens), table, page, max(lens))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    qkv, q, o, k, v = bf(n, 5120), bf(n, 32, 128), bf(n, 32, 128), bf(14, page, 4, 128), bf(14, page, 4, 128)
    stream, normed, out = res.clone(), bf(n, H), bf(n, H)
    ws, aws = m.new_prompt_workspace(n), m.new_attn_workspace()
    m.flint_linear_bf16(x, w_qkv, qkv, ws)
    m.flint_qk_norm_rope_kv_paged_bf16(qkv, gain, gain, batch, q, k, v, rope_theta=1e6)
    m.flint_attn_paged_bf16(q, k, v, batch, o, aws)
    m.flint_linear_bf16(o.view(n, 4096), w_o, stream, ws, residual=stream)
    m.flint_moe_rmsnorm_bf16(stream, normed)
    m.flint_moe_prompt_bf16(normed, stream, layer["wr"], None, layer["w13"], layer["w2"],
                            layer["ws13"], layer["ws2"], out, ws)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    p.check(qkv, p.linear(x, w_qkv, None, None, p.NONE, torch.bfloat16))
    p.check(stream, p.linear(o.view(n, 4096), w_o, None, res, p.NONE, torch.bfloat16))
    keys, vals = k.view(-1, 4, 128).double(), v.view(-1, 4, 128).double()
    at = 0
    for s, ln in enumerate(lens):
        first = [0, 9][s] * page
        kk, vv = (t[first:first + ln].repeat_interleave(8, 1) for t in (keys, vals))
        score = torch.einsum("thd,jhd->htj", q[at:at + ln].double(), kk) * 128 ** -0.5
        mask = torch.ones(ln, ln, device="cuda").triu(1).bool()
        prob = score.masked_fill(mask, float("-inf")).softmax(-1)
        want, size = (torch.einsum("htj,jhd->thd", prob, t) for t in (vv, vv.abs()))
        # A score is off by 128 fp32 additions, a weight by twice that (itself and the sum), by
        # its half step in bf16 and by 2^-16 for the exponential; then the output's half step.
        off = 144 * p.ADD * 128 ** -0.5 * torch.einsum("thd,jhd->htj", q[at:at + ln].double().abs(), kk.abs())
        err = (HALF + 2.0 ** -16 + 2 * float(off.max())) * size
        p.check(o[at:at + ln], (want, err + HALF * (want.abs() + err)))
        at += ln
    _check_layer(out, _layer_ref(normed, stream, layer, None, False))


def test_binding_refuses(ws):
    lg = torch.zeros(4, E, device="cuda")
    out = _select(ws, lg)
    for i in range(5):
        bad = list(out)
        bad[i] = bad[i][:-1].contiguous()
        with pytest.raises(m.FlintError):
            m.flint_moe_select(lg, None, *bad, ws)
    for bad in (lg.half(), lg[:, :128], lg.cpu(), lg[:0], torch.zeros(8193, E, device="cuda")):
        with pytest.raises(m.FlintError):
            m.flint_moe_select(bad, None, *out, ws)
    x = torch.zeros(4, H, dtype=torch.bfloat16, device="cuda")
    y, row = torch.zeros(24, H, dtype=torch.bfloat16, device="cuda"), out[4]
    m.flint_moe_combine_bf16(x, y, row, out[1], None, x)
    for bad in ((x, y[:23], row, out[1], None, x), (x, y, row[:3], out[1], None, x), (x, y, row, row, None, x),
                (x, y, row, out[1], x[:2], x), (x, y, row, out[1], None, x[:2]), (x.float(), y, row, out[1], None, x)):
        with pytest.raises(m.FlintError):
            m.flint_moe_combine_bf16(*bad)

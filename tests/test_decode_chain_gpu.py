"""Decode calls and paged attention right behind the library's kernels that write what they
read, which begin before those have ended: the same bits as with a wait between the calls."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests import _prompt as p
from tests.test_prompt_chain_gpu import BF, H, TURNS, _empty, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return fs.layer_weights(1001, fs.FULL, device="cuda")


@pytest.mark.parametrize("n", [1, 2, 8, 9, 40, 256])
def test_norm_then_decode(layer, n):
    g = p.gen(n)
    data, x, ws = [p.bf(g, n, H) for _ in range(TURNS)], _empty(n, H), m.new_workspace(n)

    def turn(i, wait, out):
        m.flint_moe_rmsnorm_bf16(data[i], x)
        wait()
        m.flint_moe_decode_bf16(x, data[i], layer["wr"], None, layer["w13"], layer["w2"],
                                layer["ws13"], layer["ws2"], out[0], ws)
        wait()

    _same(turn, [_empty(n, H)])
    assert m.flint_moe_get_device_status(ws) == m.FLINT_OK


def test_append_then_attend(layer):
    """Two prompts into an E4M3 cache, blocks' scales too, and at once the attention of all
    their tokens and of their last ones."""
    lens, page = [33, 70], 16
    n = sum(lens)
    g = p.gen(7)
    data = [p.bf(g, n, 5120, scale=2.0 ** (i % 7 - 3)) for i in range(TURNS)]
    gain = torch.ones(128, dtype=BF, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32(0, 1, 2, -1, -1, 3, 4, 5, 6, 7).view(2, 5)
    prompts = m.PagedBatch(i32(0, lens[0], n), i32(*lens), table, page, max(lens))
    last = m.PagedBatch(i32(0, 1, 2), i32(*lens), table, page, 1)
    code = lambda: torch.zeros(8, page, 4, 128, dtype=torch.uint8, device="cuda")  # noqa: E731
    scale = lambda: _empty(8, 1, 4, dtype=torch.float32)  # noqa: E731
    q, one, k, v, ks, vs = _empty(n, 32, 128), p.bf(g, 2, 32, 128), code(), code(), scale(), scale()
    ws = m.new_attn_workspace()

    def turn(i, wait, out):
        for batch, query, o in ((prompts, q, out[0]), (last, one, out[1])):
            m.flint_qk_norm_rope_kv_paged_fp8(data[i], gain, gain, prompts, q, k, v, ks, vs, rope_theta=1e6)
            wait()
            m.flint_attn_paged_fp8(query, k, v, ks, vs, batch, o, ws)
            wait()

    _same(turn, [_empty(n, 32, 128), _empty(2, 32, 128)])
    assert m.flint_attn_get_device_status(ws) == m.FLINT_OK

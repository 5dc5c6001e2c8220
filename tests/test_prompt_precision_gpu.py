"""The output rule of the layer's calls (max relative error 2e-2 on the output and on the
experts' part of it) for the layer of prompts, on both sides of every change of its method."""
from __future__ import annotations

import pytest
import torch

import flint_synth as fs
import moe_decode_sigmoid_gb300 as m
from tests._util import REL_TOL, TAU, rel_err, rel_err_delta
from tests.test_moe_prompt_gpu import K, _layer_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    return fs.layer_weights(1001, fs.FULL, device="cuda")


def _run(W, n, offset=None, dims=None, seed=3000, gain=1.0):
    x, res = fs.tokens(seed + n, n, device="cuda")
    W = dict(W)
    if gain != 1.0:
        W["w13"], W["ws13"] = W["w13"] * gain, W["ws13"] * gain
    ws, out = m.new_prompt_workspace(n), torch.empty_like(res)
    m.flint_moe_prompt_bf16(x, res, W["wr"], offset, W["w13"], W["w2"], W["ws13"], W["ws2"], out, ws,
                            dims=dims)
    assert m.flint_prompt_get_device_status(ws) == m.FLINT_OK
    want, _, _, _, _, gaps = _layer_ref(x, res, W, offset, dims is m.SELECT_DIMS)
    sure = gaps[:, K - 1] >= TAU
    assert int(sure.sum()) >= 0.9 * n
    got, want, res = (t[sure].double().cpu().numpy() for t in (out, want, res))
    return got, want, res


@pytest.mark.parametrize("n", [128, 129, 300, 1000, 1024, 1025, 2100, 8192])
def test_output_rule(layer, n):
    got, want, res = _run(layer, n)
    errs = rel_err(got, want), rel_err_delta(got, want, res)
    assert max(errs) <= REL_TOL, errs


@pytest.mark.parametrize("n", [200, 1500])
def test_output_rule_with_offsets(layer, n):
    """Offsets that prefer some experts, whose groups then have tiles of many rows."""
    offset = fs.logit_offsets(1003, device="cuda")
    got, want, res = _run(layer, n, offset, m.SELECT_DIMS)
    errs = rel_err(got, want), rel_err_delta(got, want, res)
    assert max(errs) <= REL_TOL, errs


@pytest.mark.parametrize("n", [200, 1100])
def test_output_rule_of_large_h(layer, n):
    """Gate and up weights 700 times as large: values of h far beyond 65504, and sums whose
    residual no longer counts."""
    got, want, res = _run(layer, n, gain=700.0)
    errs = rel_err(got, want), rel_err_delta(got, want, res)
    assert max(errs) <= REL_TOL, errs

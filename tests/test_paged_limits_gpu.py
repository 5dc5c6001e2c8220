"""GPU parity of the paged append at the ends of its ranges: rotations, rows,
sequences, pages, and what lies around the memory it writes."""
from __future__ import annotations

import pytest
import torch

from tests._paged import BLOCK, Case, D
from tests.test_paged_append_gpu import _append, _check_append, _kept, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    import moe_decode_sigmoid_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("theta", [1e-6, 1e-3, 0.5, 1.0, 1e9])
def test_rotations_of_any_theta(m, fmt, theta):
    """Below 1 a token's step is more than a turn: 8e5 rad at 1e-6, which fp64
    holds to 1e-10 and 1100 positions take to 1e-7, under the bound's 2^-17.  The
    call's theta is an fp32 number, and so the reference's has to be: 1e-3 rounded
    by 5e-8 of itself turns 900 rad a token by 4e-5."""
    theta = float(torch.tensor(theta, dtype=torch.float32))
    c = Case(701, fmt, [40, 1, 17], [1100, 33, 17])
    rows = _rows(c, 801)
    before = _kept(c)
    q = _append(m, c, *rows, theta)
    _check_append(c, *rows, theta, 1e-6, q, before)

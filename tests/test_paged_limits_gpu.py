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


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 2, 18, 32])
def test_256_sequences_that_straddle_blocks(m, fmt, new):
    """The most sequences, starting at every place in a block, 15 among them; 32
    each are the most rows."""
    c = Case(710 + new, fmt, [new] * 256, [new + (15 if i % 3 == 0 else i % 37) for i in range(256)],
             nq=2, nkv=1, rows_after=0 if new == 32 else 5)
    rows = _rows(c, 810)
    before = _kept(c)
    q = _append(m, c, *rows, 1e6)
    _check_append(c, *rows, 1e6, 1e-6, q, before)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total,page", [
    ([8192], [8192], 64), ([8192], [8207], 16), ([1] * 255 + [8192 - 255], [31] * 255 + [8000], 32),
    ([5000, 0, 3192], [5001, 70, 3207], 256)])
def test_the_most_rows(m, fmt, new, total, page):
    c = Case(720 + len(new), fmt, new, total, page=page, nq=4, nkv=2)
    rows = _rows(c, 820)
    before = _kept(c)
    q = _append(m, c, *rows, 1e6)
    _check_append(c, *rows, 1e6, 1e-6, q, before)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [128, 256, 512, 1024])
def test_large_pages(m, fmt, page):
    c = Case(730 + page, fmt, [page + 3, 1, 40], [2 * page + 5, page + 1, page], page=page, nq=8, nkv=2,
             rows_after=2)
    rows = _rows(c, 830)
    before = _kept(c)
    q = _append(m, c, *rows, 1e6)
    _check_append(c, *rows, 1e6, 1e-6, q, before)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pages_beyond_32_bits_of_bytes(m, fmt):
    """The last pages of caches of more than 2^32 bytes: the bits that a small cache
    gets, and nothing in any other page."""
    c = Case(740, fmt, [70, 1], [90, 40], page=64)
    qkv, qn, kn = _rows(c, 840)
    pages = (1 << 32) // (64 * 4 * D * (2 if fmt == "bf16" else 1)) + 40
    far = pages - c.n_pages
    big, small = [], []
    for x, s in ((c.k, c.ks), (c.v, c.vs)):
        for t in (c.shaped(x),) + ((c.scaled(s),) if fmt == "e4m3" else ()):
            y = torch.zeros((pages,) + t.shape[1:], dtype=t.dtype, device="cuda")
            y[far:] = t
            big.append(y)
            small.append(t)
    b = m.PagedBatch(c.q_start, c.kv_len, c.table + far, 64, 70)
    q = torch.empty_like(c.q)
    if fmt == "bf16":
        m.flint_qk_norm_rope_kv_paged_bf16(qkv, qn, kn, b, q, *big, 1e6)
    else:
        m.flint_qk_norm_rope_kv_paged_fp8(qkv, qn, kn, b, q, big[0], big[2], big[1], big[3], 1e6)
    assert torch.equal(_append(m, c, qkv, qn, kn, 1e6).view(torch.int16), q.view(torch.int16))
    for x, y in zip(small, big):
        assert torch.equal(y[far:].contiguous().view(torch.uint8), x.contiguous().view(torch.uint8))
        assert not y[:far].view(torch.uint8).view(torch.int64).any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_hostile_numbers_leave_what_lies_around_the_caches(m, fmt):
    """Offsets, lengths and pages outside their ranges: the memory around the queries,
    the caches and the scales, and the pages that no table names, stay as they were."""
    c = Case(750, fmt, [4, 4], [100, 60], rows_after=2, extra=3)
    qkv, qn, kn = _rows(c, 850)
    free = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    free[c.table[c.table >= 0].long()] = False
    around = []

    def guarded(t, fill):
        g = torch.full((t.shape[0] + 16,) + t.shape[1:], fill, dtype=t.dtype, device="cuda")
        g[8:-8] = t
        around.append((g, fill))
        return g[8:-8]

    q = guarded(c.q, 7.25)
    caches = [guarded(c.shaped(x), 7 if fmt == "e4m3" else 7.25) for x in (c.k, c.v)]
    scales = [guarded(c.scaled(x), 7.25) for x in (c.ks, c.vs)] if fmt == "e4m3" else []
    kept = [x.clone() for x in caches + scales]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    bad = c.table.clone()
    bad[:, 1::2] = i32([[c.n_pages], [-(1 << 31)]])
    call = m.flint_qk_norm_rope_kv_paged_bf16 if fmt == "bf16" else m.flint_qk_norm_rope_kv_paged_fp8
    most = (1 << 31) - 1
    for table in (c.table, bad):
        for q_start, kv in (([0, 4, 1 << 30], [100, 60]), ([-5, 4, 5], [100, 1 << 30]),
                            ([4, 0, -3], [-9, 60]), ([0, most, 0], [-(1 << 31), 60]),
                            ([0, 10, 0], [7, 2]), ([-most, most, most], [most, most])):
            call(qkv, qn, kn, m.PagedBatch(i32(q_start), i32(kv), table, c.page, 4), q, *caches, *scales,
                 1e6, dims=m.AttnDims(c.nq, c.nkv, D))
    torch.cuda.synchronize()
    for g, fill in around:
        assert (g[:8] == fill).all() and (g[-8:] == fill).all()
    for x, k in zip(caches + scales, kept):
        assert torch.equal(x[free].view(torch.uint8), k[free].view(torch.uint8))

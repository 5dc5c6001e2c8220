"""What the paged calls' binding refuses before it hands numbers to C, where a
32-bit field would cut them to other, valid ones."""
from __future__ import annotations

import pytest
import torch

import moe_decode_sigmoid_gb300 as m

BEYOND = [1 << 31, (1 << 32) + 1, -(1 << 32) + 5, 1 << 40]


@pytest.mark.parametrize("value", BEYOND + [0, -1])
def test_bounds_on_new_tokens_beyond_32_bits(value):
    with pytest.raises(m.FlintError) as e:
        m.PagedBatch(None, None, None, 16, value)
    assert e.value.status == m.FLINT_ERR_INVALID_ARG and "max_q_len" in str(e.value)


@pytest.mark.parametrize("value", [(1 << 32) + 16, 0, 48])
def test_page_sizes_beyond_32_bits(value):
    with pytest.raises(m.FlintError) as e:
        m.PagedBatch(None, None, None, value, 1)
    assert e.value.status == m.FLINT_ERR_INVALID_ARG and "page_size" in str(e.value)


@pytest.mark.parametrize("value", BEYOND + [-1, 512.5, "512", None])
@pytest.mark.parametrize("fp8", [False, True])
def test_windows_beyond_32_bits_or_not_whole(value, fp8):
    q = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    f, n = (m.flint_attn_paged_fp8, 4) if fp8 else (m.flint_attn_paged_bf16, 2)
    with pytest.raises(m.FlintError) as e:
        f(q, *[None] * n, "batch", q, None, window=value)
    assert e.value.status == m.FLINT_ERR_INVALID_ARG and "window" in str(e.value)


class _Table(torch.Tensor):
    """A page table of any shape that says it is on a device, without storage."""
    is_cuda = True


@pytest.mark.parametrize("columns", [(1 << 32) + 1, (1 << 23) // 16 + 1])
def test_page_tables_beyond_the_longest_sequence(columns):
    table = torch.zeros(1, 1, dtype=torch.int32).expand(1, columns)
    with pytest.raises(m.FlintError) as e:
        m.PagedBatch(None, None, table.as_subclass(_Table), 16, 1)
    assert e.value.status == m.FLINT_ERR_INVALID_ARG and "page_table" in str(e.value)


def test_arming_a_stall_wants_a_workspace():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    L, n = m.lib(), m.flint_attn_workspace_bytes()
    assert L.flint_attn_debug_arm_stall(None, n, None) == m.FLINT_ERR_WORKSPACE
    assert L.flint_attn_debug_arm_stall(0x100008, n, None) == m.FLINT_ERR_WORKSPACE
    assert L.flint_attn_debug_arm_stall(0x100000, n - 1, None) == m.FLINT_ERR_WORKSPACE
    with pytest.raises(m.FlintError):
        m.flint_attn_debug_arm_stall(torch.zeros(n, dtype=torch.uint8))

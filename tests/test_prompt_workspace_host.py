"""The bytes of a prompt workspace grow with its tokens, so that one serves every smaller call."""
from __future__ import annotations

import moe_decode_sigmoid_gb300 as m


def test_bytes_never_fall():
    from moe_decode_sigmoid_gb300 import build
    build.build()
    sizes = [m.flint_prompt_workspace_bytes(n) for n in range(m.PAGED_MAX_TOKENS + 1)]
    assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
    # what include/flint_moe.h says of them
    assert 1.5e6 < sizes[1] < 1.7e6 and 10.6e6 < sizes[128] < 10.8e6
    assert all(b <= sizes[128] + 45000 * n for n, b in enumerate(sizes) if 128 < n <= 4096)
    assert 193e6 < sizes[4096] < 194e6
    assert all(b <= max(sizes[4096], sizes[128] + 31000 * n) for n, b in enumerate(sizes) if n > 4096)

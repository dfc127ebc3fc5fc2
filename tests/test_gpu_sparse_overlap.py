"""Buffers that share memory with what the append with rotation, or attention over
lists of blocks, reads elsewhere: refused before anything is launched."""
import pytest
import torch

import bit_quantized_kv_decode_gb300 as kvq
from tests.rows_testlib import starts

pytestmark = pytest.mark.gpu


def test_windows_over_queries_and_angles():
    T, H, D = 6, 2, 128
    n = H * 128 * D
    memory = torch.zeros(6 * n, device="cuda")
    desc = kvq.cache_desc(4, 1, 0, H, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    k, v = (torch.randn(T, H, D, device="cuda") for _ in "kv")
    cu, lens = starts([T]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")

    def window(at):
        return memory[at:at + n].view(1, H, 128, D)

    table, q = memory[:40 * D].view(40, D), memory[2 * n:2 * n + T * 8 * D].view(T, 8, D)
    own = kvq.rotary_table(40, D)

    def call(angles, **kw):
        return kvq.append_rotary(desc, angles, k, v, cu, lens, *caches, max_blocks=1, **kw)

    bad = [lambda: call(table, k_window=window(0), v_window=window(3 * n)),
           lambda: call(table, k_window=window(3 * n), v_window=window(40 * D - 4)),
           lambda: call(table, k_window=window(3 * n), v_window=window(4 * n), k_window_out=window(0)),
           lambda: call(table, k_window=window(3 * n), v_window=window(4 * n), v_window_out=window(40 * D - 4)),
           lambda: call(own, q=q, k_window=window(n + 4), v_window=window(4 * n)),
           lambda: call(own, q=q, k_window=window(0), v_window=window(2 * n + T * 8 * D - 4)),
           lambda: call(own, q=q, k_window=window(0), v_window=window(4 * n), k_window_out=window(2 * n))]
    for i, wrong in enumerate(bad):
        with pytest.raises(ValueError, match="a window overlaps"):
            wrong()
            pytest.fail(f"call {i} was not refused")
    assert (memory == 0).all()
    call(own, q=q, k_window=window(n), v_window=window(2 * n + T * 8 * D))  # right before, right behind
    call(table, k_window=window(0), v_window=window(4 * n), k_window_out=window(n), v_window_out=window(5 * n))  # read by both
    assert (memory[:40 * D] == 0).all()

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


def test_workspaces_over_the_cache():
    lens = torch.tensor([200, 130], dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 1, 0, 2, 4)
    size = kvq.sparse_workspace_size(desc, 2, 8, 32)
    assert size > 0
    memory = torch.zeros(size + (1 << 18), dtype=torch.uint8, device="cuda")
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    codes = caches[0][0]
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    blocks, counts = (torch.ones(shape, dtype=torch.int32, device="cuda") for shape in ((2, 2, 32), (2, 2)))
    for i in range(6):
        for at in (0, size - 256):
            held = [list(c) for c in caches]
            t = held[i // 3][i % 3]
            held[i // 3][i % 3] = memory[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
            with pytest.raises(ValueError, match="workspace overlaps"):
                kvq.sparse_decode_attn(desc, q, *held, lens, blocks, counts, max_blocks=2, workspace=memory)
                pytest.fail(f"array {i} at {at} was not refused")
    held = memory[size:size + codes.numel()].view(codes.shape)  # behind the bytes that are used
    kvq.sparse_decode_attn(desc, q, (held, *caches[0][1:]), caches[1], lens, blocks, counts, max_blocks=2, workspace=memory)

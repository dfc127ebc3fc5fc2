"""Buffers of one call that share memory are refused where the call writes one of
them: outputs, workspaces and windows, shared in part too."""
import pytest
import torch

import bit_quantized_kv_decode_gb300 as kvq
from bit_quantized_kv_decode_gb300._lib import Rows


def test_window_ranges():
    """The check itself, on made-up addresses: windows of 4096 bytes, rows of
    2 x 2 x 64 16-bit values."""
    k, v = Rows(1 << 20, 128, 64), Rows(2 << 20, 128, 64)

    def check(kw, kwo, vw, vwo):
        kvq._windows_apart(kw, kwo, vw, vwo, 4096, k, v, 2, 2, 64, 2)

    at = 1 << 22
    check(at, at, at + 4096, at + 4096)
    check(at, at + 4096, at, at + 8192)  # only read where they are the same
    check(None, None, at, at)
    check((1 << 20) + 512, (1 << 20) + 512, (2 << 20) - 4096, (2 << 20) - 4096)  # right behind, right before the rows
    for bad in ((at, at, at + 4080, at + 4080), (at, at + 16, None, None), (None, None, at, at - 4080),
                (at, at + 4096, at + 8192, at + 4096 + 16), (at, at + 8192, at + 8192 + 4080, at + 16384),
                ((1 << 20) + 496, (1 << 20) + 496, None, None), (None, None, (2 << 20) - 4080, (2 << 20) - 4080),
                (at, at, (1 << 20) - 4080, (1 << 20) - 4080)):
        with pytest.raises(ValueError, match="overlaps|same memory"):
            check(*bad)


@pytest.mark.gpu
def test_windows_that_share_memory():
    T, H, D = 6, 2, 128
    k, v = (torch.randn(T, H, D, device="cuda") for _ in "kv")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 1, 1, H, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    n = H * 128 * D
    memory = torch.zeros(8 * n, device="cuda")

    def at(i):
        return memory[i:i + n].view(1, H, 128, D)

    rows = memory[:T * H * D].view(T, H, D)
    bad = [(k, dict(k_window=at(0), v_window=at(n - 128))), (k, dict(k_window=at(n - 128), v_window=at(0))),
           (k, dict(k_window=at(0), v_window=at(2 * n), k_window_out=at(128))),
           (k, dict(k_window=at(0), v_window=at(2 * n), v_window_out=at(2 * n - 128))),
           (k, dict(k_window=at(0), v_window=at(2 * n), k_window_out=at(n), v_window_out=at(2 * n - 128))),
           (k, dict(k_window=at(0), v_window=at(2 * n), k_window_out=at(4 * n), v_window_out=at(4 * n + 128))),
           (k, dict(k_window=at(0), v_window=at(2 * n), k_window_out=at(4 * n), v_window_out=at(128))),
           (rows, dict(k_window=at(0), v_window=at(2 * n))), (rows, dict(k_window=at(2 * n), v_window=at(128)))]
    before = [[t.clone() for t in c] for c in caches]
    for i, (x, kw) in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps|same memory"):
            kvq.append_chunk(desc, x, v, cu, lens, *caches, max_blocks=1, **kw)
            pytest.fail(f"call {i} was not refused")
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for c, d in zip(caches, before) for a, b in zip(c, d))
    for kw in (dict(k_window=at(0), v_window=at(n)), dict(k_window=at(0), v_window=at(n), k_window_out=at(2 * n)),
               dict(k_window=at(0), v_window=at(0), k_window_out=at(n), v_window_out=at(2 * n))):  # only read
        kvq.append_chunk(desc, k, v, cu, lens, *caches, max_blocks=1, **kw)


@pytest.mark.gpu
def test_outputs_and_workspaces_that_share_memory():
    T, D = 6, 128
    qkv = torch.randn(T, 12, D, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :8].contiguous(), qkv[:, 8:10], qkv[:, 10:]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 1, 1, 2, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    n = kvq.chunk_workspace_size(desc, 1, T, 8, 1)
    memory = torch.zeros(n + (1 << 20), dtype=torch.uint8, device="cuda")

    def out(i):
        return memory[i:i + T * 8 * D * 2].view(torch.bfloat16).view(T, 8, D)

    def lse(i):
        return memory[i:i + T * 8 * 4].view(torch.float32).view(T, 8)

    ws = memory[:n]
    held = memory[n - T * 8 * D * 2:n].view(torch.bfloat16).view(T, 8, D)
    bad = [lambda: kvq.prompt_attn(q, k, v, cu, out=out(0), lse=lse(0)),
           lambda: kvq.prompt_attn(q, k, v, cu, out=out(0), lse=lse(T * 8 * D * 2 - 16)),
           lambda: kvq.chunk_attn(desc, q, *caches, cu, lens, max_blocks=1, out=out(160), lse=lse(0)),
           lambda: kvq.chunk_attn(desc, q, *caches, cu, lens, max_blocks=1, out=out(n - 16), workspace=ws),
           lambda: kvq.chunk_attn(desc, q, *caches, cu, lens, max_blocks=1, lse=lse(n - 16), workspace=ws),
           lambda: kvq.chunk_attn(desc, held, *caches, cu, lens, max_blocks=1, workspace=ws)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps"):
            call()
            pytest.fail(f"call {i} was not refused")
    assert (memory == 0).all()
    kvq.prompt_attn(q, k, v, cu, out=out(0), lse=lse(T * 8 * D * 2))
    for space in (ws, memory):  # a longer workspace is used up to the call's size
        kvq.chunk_attn(desc, q, *caches, cu, lens, max_blocks=1, out=out(n), lse=lse(n + T * 8 * D * 2), workspace=space)

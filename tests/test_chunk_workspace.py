"""Workspace of chunk attention: a buffer sized for one call serves every smaller
one, whatever row shape the smaller call takes."""
import itertools

import pytest
import torch

import __graft_entry__ as entry
import bit_quantized_kv_decode_gb300 as kvq


@pytest.mark.parametrize("bits,dim,group", [(4, 128, 128), (4, 128, 32), (2, 128, 32), (4, 64, 64), (2, 64, 32),
                                            (4, 256, 64), (2, 256, 128)])
def test_never_smaller_for_a_larger_call(bits, dim, group):
    entry.build()
    desc = kvq.cache_desc(bits, 1, 0, 8, 1024, head_dim=dim, group=group)
    sizes = {(b, t, h): kvq.chunk_workspace_size(desc, b, t, h, 64)
             for b in (1, 2, 64, 4096) for t in (1, 32, 512, 2000, 65536) for h in (8, 32, 128)}
    for (large, n), (small, m) in itertools.product(sizes.items(), repeat=2):
        if all(a >= b for a, b in zip(large, small)):
            assert n >= m, (large, n, small, m)


@pytest.mark.gpu
def test_a_buffer_for_many_sequences_serves_one():
    from tests.test_gpu_chunk_attn import Setup
    wide = Setup(4, (1, 0), 128, 128, 2, 4, new=(3,) * 40, total=(50,) * 40, seed=31)
    one = Setup(4, (1, 0), 128, 128, 2, 4, new=(100,), total=(700,), seed=32)
    ws = torch.empty(kvq.chunk_workspace_size(wide.desc, 40, 120, 8, 8), dtype=torch.uint8, device="cuda")
    for s in (wide, one, wide):
        want, want_lse = s.call()
        got, got_lse = s.call(workspace=ws)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)

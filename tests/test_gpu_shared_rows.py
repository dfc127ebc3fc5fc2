"""Sequences that share rows behind a decreasing entry of cu_seqlens: the call is
reported, what it writes is right, and nothing else is written.  (Rows may be
left as they were: the launch is made for sequences that do not overlap.)"""
import pytest
import torch

from tests.rows_testlib import starts
from tests.test_gpu_prompt_attn import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T,dim", [(300, 64), (4000, 128), (2500, 256)])
@pytest.mark.parametrize("times", [2, 5])
def test_prompts(causal, T, dim, times):
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(T + 60, 4, 1, dim, torch.bfloat16, seed=41)
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device="cuda")
    kvq.prompt_attn(q, k, v, cu, causal=causal, out=out, dev_status=status)
    assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN
    alone = kvq.prompt_attn(q[:T], k[:T], v[:T], starts([T]).cuda(), causal=causal)
    same = (out[:T] == alone).flatten(1).all(1)
    left = (out[:T] == 7.0).flatten(1).all(1)
    assert (same | left).all() and same.any() and (out[T:] == 7.0).all()


@pytest.mark.parametrize("T", [100, 5000])
@pytest.mark.parametrize("schemes", [(0, 0), (1, 1)])
def test_append(T, schemes):
    import bit_quantized_kv_decode_gb300 as kvq
    wide, B = (T + 127) // 128 + 1, 5
    desc = kvq.cache_desc(4, *schemes, 2, B * wide)
    g = torch.Generator(device="cuda").manual_seed(42)
    k, v = (torch.randn(T + 9, 2, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(batch, cu):
        caches = [kvq.alloc_cache(desc) for _ in "kv"]
        for c in caches:
            for t in c:
                t.view(torch.uint8).fill_(0xA7)
        windows = [torch.zeros(batch, 2, 128, 128, device="cuda") for _ in "kv"]
        kvq.append_chunk(desc, k, v, cu, torch.zeros(batch, dtype=torch.int32, device="cuda"), *caches, *windows,
                         max_blocks=wide, dev_status=status)
        return [t.view(torch.uint8).view(B, wide, -1) for c in caches for t in c]

    got = call(B, torch.tensor([0, T] * 3, dtype=torch.int32, device="cuda"))
    assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN
    alone = call(1, starts([T]).cuda())
    for a, b in zip(got, alone):
        for s in (0, 2, 4):
            same, left = (a[s] == b[0]).all(1), (a[s] == 0xA7).all(1)
            assert (same | left).all()
        assert (a[1] == 0xA7).all() and (a[3] == 0xA7).all()

"""The prompt side and decode together, as a serving program runs them: a
first chunk by prompt attention on its raw rows, written to the cache, later
chunks and drafted tokens by chunk attention over the cache, then decode
steps; each step against the definition in 64 bits."""
import math

import pytest
import torch

import kvq_synth as synth
from tests.rows_testlib import HALF_STEP, assert_rows_close, attend64, cache_values, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,schemes,dim,group", [(4, (1, 0), 128, 128), (2, (0, 1), 64, 32), (4, (1, 1), 256, 64)])
def test_prompt_chunks_drafts_and_decode(bits, schemes, dim, group):
    import bit_quantized_kv_decode_gb300 as kvq
    hkv, per, B, wide = 2, 4, 2, 6
    g = torch.Generator(device="cuda").manual_seed(bits + dim)
    table, pages = synth.page_table_for(torch.tensor([wide * 128] * B), 3, wide)
    pt = table.cuda()
    desc = kvq.cache_desc(bits, *schemes, hkv, pages, head_dim=dim, group=group)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    windows = [torch.zeros(B, hkv, 128, dim, device="cuda") for _ in "kv"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [0, 0]
    scale = 1.0 / math.sqrt(dim)
    for step, new in enumerate(([150, 260], [130, 7], [4, 4], [200, 1])):
        T = sum(new)
        qkv = torch.randn(T, (per + 2) * hkv, dim, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv[:, :per * hkv], qkv[:, per * hkv:(per + 1) * hkv], qkv[:, (per + 1) * hkv:]
        cu = starts(new).cuda()
        before = torch.tensor(held, dtype=torch.int32, device="cuda")
        outs = [torch.zeros_like(w) for w in windows]
        kvq.append_chunk(desc, k, v, cu, before, *caches, *windows, page_table=pt, k_window_out=outs[0],
                         v_window_out=outs[1], dev_status=status)
        after = before + (cu[1:] - cu[:-1])
        total = after.tolist()
        if step == 0:  # the first chunk is the whole sequence so far: its raw rows
            out = kvq.prompt_attn(q, k, v, cu, dev_status=status)
        else:
            out = kvq.chunk_attn(desc, q, *caches, cu, after, pt, dev_status=status)
        assert int(status.item()) == 0
        kk, vv = (cache_values([t.cpu() for t in caches[w]], total, bits, w, schemes[w], table, dim) for w in (0, 1))
        a = 0
        for b, n in enumerate(new):
            rows = slice(a, a + n)
            a += n
            if step == 0:
                ref, _, tol, _ = attend64(q[rows], k[rows], v[rows], 0, True, scale, HALF_STEP[torch.bfloat16])
            else:
                ref, _, tol, _ = attend64(q[rows], kk[b, :total[b]].cuda(), vv[b, :total[b]].cuda(), total[b] - n, True,
                                          scale, HALF_STEP[torch.float16])
            assert_rows_close(out[rows], ref, tol, q.dtype, f"step {step}, sequence {b}")
        if step == 2:  # two of the four drafted tokens are rejected: write again from the old windows
            keep = starts([2, 2]).cuda()
            rows = torch.tensor([0, 1, 4, 5], device="cuda")
            kvq.append_chunk(desc, k[rows], v[rows], keep, before, *caches, *windows, page_table=pt,
                             dev_status=status)
            held = [h + 2 for h in held]
        else:
            windows = outs
            held = total
    # decode steps on the cache that the chunks left
    lens = torch.tensor(held, dtype=torch.int32, device="cuda")
    for _ in range(3):
        x = [torch.randn(B, hkv, dim, generator=g, device="cuda") for _ in "kv"]
        for w in (0, 1):
            kvq.append(desc, w, x[w], lens, caches[w], windows[w], page_table=pt, dev_status=status)
        lens += 1
        held = [h + 1 for h in held]
        q = torch.randn(B, per * hkv, dim, generator=g, device="cuda").to(torch.bfloat16)
        out, _ = kvq.decode_attn(desc, q, *caches, lens, pt, mode=kvq.OPERANDS_BF16, dev_status=status)
        assert int(status.item()) == 0
        kk, vv = (cache_values([t.cpu() for t in caches[w]], held, bits, w, schemes[w], table, dim, rounded=False)
                  for w in (0, 1))
        for b in range(B):
            ref = attend64(q[b:b + 1], kk[b, :held[b]].cuda(), vv[b, :held[b]].cuda(), held[b] - 1, True, scale, 0.0)[0]
            rms = ref.pow(2).mean().sqrt()
            assert (out[b].double() - ref[0]).abs().max() <= 2e-3 * rms * 4

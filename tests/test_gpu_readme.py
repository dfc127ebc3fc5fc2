"""The README's example, run as it stands, and decode steps behind it: the cache
equals the oracle's pack of the whole sequences."""
import os
import re

import numpy as np
import pytest
import torch

import kvq_synth as synth
from oracle import kvq_oracle as orc
from tests.conftest import ROOT
from tests.rows_testlib import starts

pytestmark = pytest.mark.gpu


def example():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "append_chunk" in b)


def check_cache(cache, x, lens, bits, which, scheme, table, pages):
    """The cache against the oracle's pack of x[b] ([tokens, heads, channels])."""
    wide, (hkv, dim) = table.shape[1], x[0].shape[1:]
    pad = np.zeros((len(lens), hkv, wide * 128, dim), np.float32)
    for b, n in enumerate(lens):
        pad[b, :, :n] = x[b].transpose(0, 1).cpu().numpy()
    ref = orc.pack_cache(pad, lens, bits, scheme, which, table.numpy(), pages)
    used = sorted(int(table[b, j]) for b, n in enumerate(lens) for j in range((n + 127) // 128))
    for name, got, want in zip(("codes", "scale", "zero"), cache, ref):
        got = got.cpu().view(torch.uint8 if name == "codes" else torch.int16).numpy()
        assert np.array_equal(got[used], (want if name == "codes" else want.view(np.int16))[used]), (name, which)


@pytest.mark.parametrize("schemes", [(1, 0), (0, 0), (0, 1), (1, 1)])
def test_example_then_decode_steps(schemes):
    import bit_quantized_kv_decode_gb300 as kvq
    per, hkv, dim, B, bits, wide = 4, 2, 128, 2, 4, 4
    g = torch.Generator(device="cuda").manual_seed(9)
    table, pages = synth.page_table_for(torch.tensor([wide * 128] * B), 3, wide)
    desc = kvq.cache_desc(bits, *schemes, hkv, pages)
    names = dict(kvq=kvq, desc=desc, table=table.cuda(), lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 kc=kvq.alloc_cache(desc), vc=kvq.alloc_cache(desc),
                 k_window=torch.zeros(B, hkv, 128, dim, device="cuda"), v_window=torch.zeros(B, hkv, 128, dim, device="cuda"))
    x = [[[] for _ in range(B)] for _ in "kv"]  # rows of K and V by sequence
    for suffix, new in (("", [150, 260]), ("2", [130, 7])):
        for name, heads in (("q", per * hkv), ("k", hkv), ("v", hkv)):
            names[name + suffix] = torch.randn(sum(new), heads, dim, generator=g, device="cuda").to(torch.bfloat16)
        names["cu" + suffix] = starts(new).cuda()
        for which, name in enumerate("kv"):
            for b, part in enumerate(names[name + suffix].float().split(new)):
                x[which][b].append(part)
    exec(example(), names)
    lens, caches = names["lens"], (names["kc"], names["vc"])
    assert lens.tolist() == [280, 267] and torch.isfinite(names["out"]).all() and torch.isfinite(names["out2"]).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(4):
        if step:
            for which, window in enumerate((names["k_window"], names["v_window"])):
                row = torch.randn(B, hkv, dim, generator=g, device="cuda")
                kvq.append(desc, which, row, lens, caches[which], window, page_table=names["table"], dev_status=status)
                for b in range(B):
                    x[which][b].append(row[b:b + 1])
            lens += 1
        for which in (0, 1):
            check_cache(caches[which], [torch.cat(r) for r in x[which]], lens.tolist(), bits, which, schemes[which],
                        table, pages)
    assert int(status.item()) == 0


@pytest.mark.parametrize("bits", [2, 4])
def test_without_a_window_single_tokens_go_on_as_chunks_of_one(bits):
    """What the README says of a token-wise cache that keeps no window."""
    import bit_quantized_kv_decode_gb300 as kvq
    hkv, dim, B, wide = 2, 128, 2, 3
    g = torch.Generator(device="cuda").manual_seed(10)
    table, pages = synth.page_table_for(torch.tensor([wide * 128] * B), 4, wide)
    desc = kvq.cache_desc(bits, 0, 0, hkv, pages)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = [[[] for _ in range(B)] for _ in "kv"]
    for new in ([126, 200], [1, 1], [1, 1], [1, 1]):
        rows = [torch.randn(sum(new), hkv, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
        kvq.append_chunk(desc, *rows, starts(new).cuda(), lens, *caches, page_table=table.cuda())
        lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        for which in (0, 1):
            for b, part in enumerate(rows[which].float().split(new)):
                x[which][b].append(part)
            check_cache(caches[which], [torch.cat(r) for r in x[which]], lens.tolist(), bits, which, 0, table, pages)

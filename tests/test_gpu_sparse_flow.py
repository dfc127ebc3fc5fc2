"""A serving loop over part of the cache: prompts turned by their positions and
written to the cache, attention over the turned rows, then decode steps that turn
and append a token, select blocks and attend to those; each call against the
definition in 64 bits, and the same steps from one captured graph."""
import math
import os
import re

import pytest
import torch

import kvq_synth as synth
from tests.conftest import ROOT
from tests.rows_testlib import HALF_STEP, assert_rows_close, attend64, starts
from tests.sparse_testlib import Cache, assert_sparse_close, attend_lists64, scores64, select64

pytestmark = pytest.mark.gpu


class Served(Cache):
    """Empty caches and windows that a loop fills."""

    def __init__(self, bits, schemes, hkv, dim, group, batch, wide, seed):
        import bit_quantized_kv_decode_gb300 as kvq
        self.bits, self.schemes, self.hkv, self.dim, self.group, self.wide = bits, schemes, hkv, dim, group, wide
        self.lengths = [0] * batch
        self.table_host, self.pages = synth.page_table_for(torch.tensor([wide * 128] * batch), seed, wide)
        self.table = self.table_host.cuda()
        self.desc = kvq.cache_desc(bits, *schemes, hkv, self.pages, head_dim=dim, group=group)
        self.k, self.v = (kvq.alloc_cache(self.desc) for _ in "kv")
        self.window = [torch.zeros(batch, hkv, 128, dim, device="cuda") for _ in "kv"]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.generator = torch.Generator(device="cuda").manual_seed(seed)

    def rows(self, tokens, per):
        x = torch.randn(tokens, (per + 2) * self.hkv, self.dim, generator=self.generator, device="cuda").to(torch.bfloat16)
        return x[:, :per * self.hkv], x[:, per * self.hkv:(per + 1) * self.hkv], x[:, (per + 1) * self.hkv:]


def turned64(x, angles, interleaved):
    x, angles = x.double(), angles.double()
    R = angles.shape[1]
    c, s = angles[:, None, :R // 2], angles[:, None, R // 2:]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = x.clone()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def assert_turned(got, x, angles, interleaved):
    """Three roundings in fp32 of sums of two products, then one to bf16."""
    ref = turned64(x, angles, interleaved)
    size = turned64(x.abs(), torch.cat([angles[:, :angles.shape[1] // 2].abs(), -angles[:, angles.shape[1] // 2:].abs()], 1), interleaved)
    size = torch.maximum(size.abs(), turned64(x.abs(), angles.abs(), interleaved).abs())
    bound = 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -24 * size
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("bits,schemes,dim,group,rotary,interleaved", [
    (4, (1, 0), 128, 128, 128, False), (2, (1, 1), 64, 32, 32, True), (4, (1, 0), 256, 64, 64, False)])
def test_prompt_then_decode_over_selected_blocks(bits, schemes, dim, group, rotary, interleaved):
    import bit_quantized_kv_decode_gb300 as kvq
    hkv, per, budget = 2, 4, 4
    new = [900, 127, 1, 1400]
    B, T = len(new), sum(new)
    c = Served(bits, schemes, hkv, dim, group, B, 12, bits + dim)
    table = kvq.rotary_table(12 * 128, rotary)
    q, k, v = c.rows(T, per)
    cu = starts(new).cuda()
    k_out = torch.empty(T, hkv, dim, dtype=torch.bfloat16, device="cuda")
    turned = kvq.append_rotary(c.desc, table, k, v, cu, c.lens, c.k, c.v, *c.window, page_table=c.table, interleaved=interleaved,
                               q=q, k_out=k_out, dev_status=c.status)
    out = kvq.prompt_attn(turned, k_out, v, cu, dev_status=c.status)
    c.lens += cu[1:] - cu[:-1]
    angles = table[torch.cat([torch.arange(n) for n in new]).cuda()]
    assert_turned(turned, q, angles, interleaved)
    assert_turned(k_out, k, angles, interleaved)
    a = 0
    for n in new:
        rows = slice(a, a + n)
        a += n
        ref, _, tol, _ = attend64(turned[rows], k_out[rows], v[rows], 0, True, 1.0 / math.sqrt(dim), HALF_STEP[torch.bfloat16])
        assert_rows_close(out[rows], ref, tol, q.dtype, f"prompt of {n}")

    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    static = [torch.empty(B, h, dim, dtype=torch.bfloat16, device="cuda") for h in (per * hkv, hkv, hkv)]

    def step(q, k, v):
        """One token for each: the program's own decode step, attention to a part of the cache in place of all of it."""
        qt = kvq.append_rotary(c.desc, table, k, v, one, c.lens, c.k, c.v, *c.window, page_table=c.table,
                               interleaved=interleaved, q=q, dev_status=c.status)
        c.lens.add_(1)
        blocks, counts = kvq.select_blocks(c.desc, qt, c.k, c.lens, budget, page_table=c.table, dev_status=c.status)
        out, lse = kvq.sparse_decode_attn(c.desc, qt, c.k, c.v, c.lens, blocks, counts, c.table, return_lse=True, dev_status=c.status)
        return qt, blocks, counts, out, lse

    graph = None
    for i in range(4):  # the second sequence goes over the end of its block with the first two tokens
        x = c.rows(B, per)
        if i < 2:
            qt, blocks, counts, out, lse = step(*x)
        else:
            for t, y in zip(static, x):
                t.copy_(y)
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    result = step(*static)
            graph.replay()
            qt, blocks, counts, out, lse = result
        c.lengths = [n + i + 1 for n in new]
        assert int(c.status.item()) == 0 and c.lens.tolist() == c.lengths
        assert_turned(qt, x[0], table[(c.lens - 1).long()], interleaved)
        lists = [[select64(row, budget, 1, 1) for row in score] for score in scores64(c, qt)]
        got = [[blocks[b, h, :counts[b, h]].tolist() for h in range(hkv)] for b in range(B)]
        assert got == lists
        assert_sparse_close(out, lse, *attend_lists64(c, qt, lists))
    whole, counts = kvq.select_blocks(c.desc, qt, c.k, c.lens, c.wide, page_table=c.table)
    out, lse = kvq.sparse_decode_attn(c.desc, qt, c.k, c.v, c.lens, whole, counts, c.table, return_lse=True)
    assert counts.tolist() == [[(n + 127) // 128] * hkv for n in c.lengths]
    want, want_lse = kvq.decode_attn(c.desc, qt, c.k, c.v, c.lens, c.table)
    rms = want.square().mean().sqrt()
    assert ((out.float() - want).abs() <= 3e-2 * rms + 2.0 ** -8 * (want.abs() + 3e-2 * rms)).all()
    assert ((lse - want_lse).abs() <= 1e-2).all()


def test_readme_example():
    import bit_quantized_kv_decode_gb300 as kvq
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    example = next(b for b in blocks if "select_blocks" in b)
    B, hkv, per = 3, 2, 4
    c = Served(4, (1, 0), hkv, 128, 128, B, 8, 5)
    q, k, v = c.rows(B * 600, per)
    table = kvq.rotary_table(8 * 128, 128)
    kvq.append_rotary(c.desc, table, k, v, starts([600] * B).cuda(), c.lens, c.k, c.v, *c.window, page_table=c.table)
    c.lens += 600
    q, k, v = c.rows(B, per)
    names = dict(kvq=kvq, desc=c.desc, positions=8 * 128, q=q, k=k, v=v, lens=c.lens, kc=c.k, vc=c.v, k_window=c.window[0],
                 v_window=c.window[1], table=c.table, budget=3, one_each=torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    exec(example, names)
    c.lengths = [601] * B
    assert c.lens.tolist() == c.lengths
    assert_turned(names["turned"], q, table[torch.full((B,), 600)], False)
    lists = [[select64(row, 3, 1, 1) for row in score] for score in scores64(c, names["turned"])]
    assert names["blocks"].tolist() == lists and (names["counts"] == 3).all()
    assert_sparse_close(names["out"], None, *attend_lists64(c, names["turned"], lists))

"""Prompt attention, values of V that are not finite: they reach every row that
sees their token, whatever the mask and the number of tokens, and no other row
or channel."""
import math

import pytest
import torch

from tests.rows_testlib import DTYPES, starts
from tests.test_gpu_prompt_attn import make

pytestmark = pytest.mark.gpu


def expect(out, clean, rows, heads, channel, bad):
    """out has `bad` at [rows, heads, channel], and equals clean elsewhere."""
    hit = out[rows, heads, channel]
    assert (torch.isnan(hit) if math.isnan(bad) else hit == bad).all()
    rest = out.clone()
    rest[rows, heads, channel] = clean[rows, heads, channel]
    assert torch.equal(rest, clean)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,at", [(1, 0), (100, 0), (100, 50), (100, 99), (200, 127), (200, 128), (200, 190), (256, 130),
                                  (300, 299), (513, 512)])
def test_without_a_mask_every_row_sees_them(dim, dtype, bad, n, at):
    """The second of three sequences: its last key tile is whole, or cut short
    by the next sequence."""
    import bit_quantized_kv_decode_gb300 as kvq
    lens = [70, n, 40]
    q, k, v = make(sum(lens), 8, 2, dim, DTYPES[dtype], seed=21)
    cu = starts(lens).cuda()
    clean = kvq.prompt_attn(q, k, v, cu, causal=False)
    v = v.clone()
    v[70 + at, 1, 9] = bad
    out = kvq.prompt_attn(q, k, v, cu, causal=False)
    expect(out, clean, slice(70, 70 + n), slice(4, 8), 9, bad)


def test_without_a_mask_opposite_infinities_are_not_a_number():
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(100, 4, 1, 128, torch.bfloat16, seed=22)
    clean = kvq.prompt_attn(q, k, v, starts([100]).cuda(), causal=False)
    v = v.clone()
    v[10, 0, 3], v[80, 0, 3] = math.inf, -math.inf
    expect(kvq.prompt_attn(q, k, v, starts([100]).cuda(), causal=False), clean, slice(0, 100), slice(0, 4), 3, math.nan)

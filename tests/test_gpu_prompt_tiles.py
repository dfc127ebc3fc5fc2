"""Prompt attention, causal, head dim 256: tiles of an odd number of tokens, some
of which begin at the last token of a key tile."""
import math

import pytest
import torch

from tests.rows_testlib import starts
from tests.test_gpu_prompt_attn import make
from tests.test_gpu_prompt_values import expect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("per,first", [(5, 2175), (6, 1407), (11, 1023), (13, 639), (14, 639)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("behind", [1, 5])
def test_the_next_key_tile_does_not_reach_a_tiles_first_row(per, first, bad, behind):
    import bit_quantized_kv_decode_gb300 as kvq
    assert first % (128 // per) == 0 and first % 128 == 127  # a row tile of 128 // per tokens begins there
    T = first + 200
    q, k, v = make(T, per, 1, 256, torch.bfloat16, seed=per)
    cu = starts([T]).cuda()
    clean = kvq.prompt_attn(q, k, v, cu)
    v = v.clone()
    v[first + behind, 0, 200] = bad
    out = kvq.prompt_attn(q, k, v, cu)
    expect(out, clean, slice(first + behind, T), slice(0, per), 200, bad)

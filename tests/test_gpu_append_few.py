"""Appends with no more tokens than sequences, some of them with several: blocks
that such sequences go on into, windows of those without new tokens, and entries
that are refused."""
import random

import pytest
import torch

from tests.rows_testlib import DTYPES
from tests.test_gpu_append_chunk import Setup

pytestmark = pytest.mark.gpu


def rotary_call(s, **kw):
    """append_rotary by angles of zero: every row as it is, exactly (x 1 - y 0)."""
    import bit_quantized_kv_decode_gb300 as kvq
    dim = s.rows[0].shape[2]
    table = torch.cat([torch.ones(s.wide * 128, dim // 2), torch.zeros(s.wide * 128, dim // 2)], 1).cuda()
    args = dict(k_window=s.window[0], v_window=s.window[1], page_table=s.table_dev, max_blocks=s.wide, dev_status=s.status)
    kvq.append_rotary(s.desc, table, s.rows[0], s.rows[1], s.cu, s.lens, *s.cache, **{**args, **kw})
    torch.cuda.synchronize()


# tokens before -> new ones, never more than one for each sequence in all: the
# last token of a block, both sides of it, whole blocks, and many without any
FEW = [([127, 5, 128, 126, 0, 60, 300, 0, 127, 255], [2, 0, 0, 3, 1, 0, 0, 0, 2, 1]),
       ([127, 40], [2, 0]), ([40, 127], [0, 2]), ([0, 77, 128], [0, 0, 3]),
       ([100] + [127] * 9 + [50] * 290, [270] + [2] * 9 + [0] * 290),
       ([50] * 290 + [127] * 9 + [100], [0] * 290 + [1] * 9 + [285]),
       ([64, 128] * 80 + [0] * 8, [1] * 160 + [0] * 7 + [8])]


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("case", range(len(FEW)))
@pytest.mark.parametrize("schemes,dtype,dim,group", [((1, 0), "bf16", 128, 128), ((0, 1), "fp32", 64, 32), ((1, 1), "fp16", 256, 64)])
def test_as_many_sequences_as_tokens(case, schemes, dtype, dim, group, rotary):
    old, new = FEW[case]
    assert sum(new) <= len(old)
    s = Setup(4 if dim > 64 else 2, schemes, dim, group, 2, DTYPES[dtype], True, case + 1, old, new)
    call = rotary_call if rotary else Setup.call
    outs = [torch.full_like(w, 9.0) for w in s.window]
    call(s, k_window_out=outs[0], v_window_out=outs[1])
    s.check(outs)
    call(s)  # again, the windows in place
    s.check(s.window)


@pytest.mark.parametrize("rotary", [False, True])
def test_refused_entries_among_them(rotary):
    import bit_quantized_kv_decode_gb300 as kvq
    rng = random.Random(3)
    old = [rng.choice([126, 127, 128, 60, 0]) for _ in range(40)]
    new = [0] * 40
    for b, n in ((3, 1), (7, 3), (11, 4), (20, 1), (33, 9), (39, 2)):
        new[b] = n
    old[7] = old[11] = old[39] = 127
    s = Setup(4, (1, 0), 128, 128, 2, torch.bfloat16, True, 5, old, new)
    s.lens[3], s.lens[0], s.lens[20] = -1, -7, s.wide * 128
    (rotary_call if rotary else Setup.call)(s)
    assert int(s.status.item()) == kvq.DEV_BAD_SEQ_LEN
    s.status.zero_()
    for b in (0, 3, 20):
        s.total[b] = s.old[b]
        s.x = [[t[:n] for t, n in zip(x, s.total)] for x in s.x]
    s.check(s.window)


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp32", 64), ("fp16", 256)])
@pytest.mark.parametrize("tokens", [1, 2, 9, 17])
def test_chunks_that_start_at_every_place(rotary, dtype, dim, tokens):
    """Begun blocks of every length up to some warps' tokens, and up to the block's end."""
    s = Setup(4, (1, 1), dim, 64, 2, DTYPES[dtype], True, tokens, list(range(33)) + list(range(110, 129)), [tokens] * 52)
    (rotary_call if rotary else Setup.call)(s)
    s.check(s.window)

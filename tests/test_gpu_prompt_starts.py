"""Prompt attention: entries of cu_seqlens that are out of range or go back are
reported wherever they stand, with and without a mask."""
import pytest
import torch

from tests.rows_testlib import starts
from tests.test_gpu_prompt_attn import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal,batch,at", [(False, 64, 40), (False, 33, 33), (False, 2000, 1999), (True, 320, 300),
                                             (True, 257, 257), (True, 200, 150)])
@pytest.mark.parametrize("kind", ["past the end", "negative", "back"])
def test_reported_behind_the_first_32(causal, batch, at, kind):
    import bit_quantized_kv_decode_gb300 as kvq
    lens = [3] * batch
    q, k, v = make(sum(lens), 4, 1, 64, torch.bfloat16, seed=batch)
    cu = starts(lens)
    good = [b for b in range(batch) if b not in (at - 1, at)]
    if kind == "past the end":
        cu[at:] = sum(lens) + 1
        good = list(range(at - 1))
    elif kind == "negative":
        cu[at] = -7
    else:
        cu[at] = cu[at - 1] - 1  # the sequence before it is bad, the one behind it has rows of others
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = kvq.prompt_attn(q, k, v, starts(lens).cuda(), causal=causal, dev_status=status)
    assert int(status.item()) == 0
    out = torch.full_like(q, 7.0)
    kvq.prompt_attn(q, k, v, cu.cuda(), causal=causal, out=out, dev_status=status)
    assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN
    if kind != "back":
        rows = torch.cat([torch.arange(3 * b, 3 * b + 3) for b in good]).cuda()
        assert torch.equal(out[rows], want[rows])
        left = torch.ones(len(q), dtype=torch.bool, device="cuda")
        left[rows] = False
        assert (out[left] == 7.0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_reported_where_no_sequence_is_good(causal):
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(40, 4, 1, 64, torch.bfloat16, seed=5)
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attn(q, k, v, torch.tensor([-1, 50, 41], dtype=torch.int32, device="cuda"), causal=causal, out=out,
                    dev_status=status)
    assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN and (out == 7.0).all()

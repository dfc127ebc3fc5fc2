"""Decode attention over lists of blocks: queries that are not numbers, and lists
of which every token has to count once."""
import math
import random

import pytest
import torch

from tests.sparse_testlib import Cache, as_lists

pytestmark = pytest.mark.gpu


def call(cache, q, blocks, counts):
    import bit_quantized_kv_decode_gb300 as kvq
    out, lse = kvq.sparse_decode_attn(cache.desc, q, cache.k, cache.v, cache.lens, blocks, counts, cache.table, cache.wide,
                                      return_lse=True, dev_status=cache.status)
    assert int(cache.status.item()) == 0
    return out, lse


@pytest.mark.parametrize("sequences,list_len", [(160, 2), (20, 6), (1, 300)])  # one range per list, two, more than eight
@pytest.mark.parametrize("schemes,per", [((1, 0), 4), ((0, 1), 8), ((0, 0), 2)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_queries_that_are_not_numbers(sequences, list_len, schemes, per, value):
    """A NaN or an infinity in q makes every weight of its head NaN (an infinite score less the largest one), in
    however many ranges the list is cut; the other heads are what they were."""
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, schemes, 8, [128 * list_len - 3] * sequences, seed=per)
    assert (kvq.sparse_workspace_size(c.desc, sequences, 8 * per, list_len) == 0) == (sequences == 160)
    q = c.queries(per)
    blocks, counts = as_lists([[list(range(list_len))] * 8] * sequences, list_len, 8)
    want, want_lse = call(c, q, blocks, counts)
    bad = torch.zeros(sequences, 8 * per, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[-1, 8 * per - 1] = bad[sequences // 2, per] = True
    q[:, :, 5][bad] = value
    out, lse = call(c, q, blocks, counts)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("schemes", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dim,group,per", [(64, 32, 4), (128, 128, 4), (128, 64, 8), (256, 64, 1), (256, 128, 8)])
def test_every_token_counts_once(bits, schemes, dim, group, per):
    """With q = 0 every score is 0 exactly: lse is the logarithm of the number of tokens, the output their mean.

    A lost or a repeated token changes lse by 1 / n (1.1e-5 at the most tokens here).  The sum of n ones is exact; a
    range's logarithm is off by 2 ulp of log2 n < 16 (2^-19), times ln 2; the merge adds some roundings of numbers
    below 16 (2^-21 each): 2^-18 in all.

    A probability of 1 times an fp16 scale has 11 significant bits, which the three 4-bit parts hold; products and
    sums in fp32 are allowed 2^-14 of the mean magnitude of code times scale and of the offset; then the output's
    rounding to bf16."""
    lens = [90_000, 33_333, 2_050, 128, 1]
    c = Cache(bits, schemes, 1, lens, dim, group, seed=bits + dim + per)
    rng = random.Random(dim + per)
    lists = []
    for n in lens:
        nb = (n + 127) // 128
        x = rng.sample(range(nb), max(1, nb - 3))
        lists.append([x if nb - 1 in x else x[:-1] + [nb - 1]])  # (the ragged last block among them)
    blocks, counts = as_lists(lists, max(len(x[0]) for x in lists), 1)
    q = torch.zeros(len(lens), per, dim, dtype=torch.bfloat16, device="cuda")
    out, lse = call(c, q, blocks, counts)
    v = c.values(1)
    for b, n in enumerate(lens):
        at = [t for j in lists[b][0] for t in range(j * 128, min(n, j * 128 + 128))]
        assert (lse[b].double().cpu() - math.log(len(at))).abs().max() <= 2.0 ** -18
        assert 0.5 / len(at) > 2.0 ** -18
        x = v[b, at, 0]
        ref, size = x.mean(0), x.abs().mean(0) + 2 * x.abs().max()  # |code s| <= |x| + |z|, |z| <= the largest value
        bound = 2.0 ** -14 * size + 2.0 ** -8 * (ref.abs() + 2.0 ** -14 * size)
        err = (out[b].double().cpu() - ref).abs()
        assert (err <= bound).all(), f"{n} tokens: off by {err.max().item():.3e}, {(err / bound).max().item():.2f} of the bound"

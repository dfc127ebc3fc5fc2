"""Decode attention over lists of blocks against the definition in 64 bits."""
import math
import random

import pytest
import torch

from tests.sparse_testlib import Cache, as_lists, assert_sparse_close, attend_lists64

pytestmark = pytest.mark.gpu


def some_lists(cache, most, seed, order=True):
    rng = random.Random(seed)
    lists = []
    for n in cache.lengths:
        nb = (n + 127) // 128
        of = []
        for _ in range(cache.hkv):
            x = rng.sample(range(nb), rng.randint(0, min(nb, most)))
            of.append(sorted(x) if order else x)
        lists.append(of)
    return lists


def call(cache, q, lists, list_len, expect=0, **kw):
    import bit_quantized_kv_decode_gb300 as kvq
    blocks, counts = as_lists(lists, list_len, cache.hkv)
    r = kvq.sparse_decode_attn(cache.desc, q, cache.k, cache.v, cache.lens, blocks, counts, cache.table, cache.wide,
                               return_lse=True, dev_status=cache.status, **kw)
    assert int(cache.status.item()) == expect
    return r


LENS = [1, 128, 129, 2047, 2048, 300, 3000, 5000, 777, 0]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("schemes", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("per", [4, 8])
def test_geometries(bits, schemes, dim, group, per):
    c = Cache(bits, schemes, 2, LENS, dim, group, seed=bits + dim + group + per)
    q = c.queries(per)
    lists = some_lists(c, 12, dim + group)
    lists[7] = [list(range(40)), [39]]
    assert_sparse_close(*call(c, q, lists, 40), *attend_lists64(c, q, lists))


@pytest.mark.parametrize("per", [1, 2])
@pytest.mark.parametrize("paged", [False, True])
def test_few_heads_and_any_order(per, paged):
    c = Cache(4, (1, 0), 3, LENS, paged=paged, seed=per)
    q = c.queries(per)
    lists = some_lists(c, 40, 1, order=False)
    assert_sparse_close(*call(c, q, lists, 40), *attend_lists64(c, q, lists))


@pytest.mark.parametrize("scale", [0.03, 0.3])
def test_scale_and_repeated_blocks(scale):
    c = Cache(4, (1, 0), 2, [2000, 1000], seed=3, loud=False)
    q = c.queries(4)
    lists = [[[3, 3, 15, 0, 15, 15], [15]], [[7, 7], [1, 1, 1]]]
    assert_sparse_close(*call(c, q, lists, 6, sm_scale=scale), *attend_lists64(c, q, lists, scale), scale * math.sqrt(128))


def test_one_range_per_list():
    """So many lists that each is one CTA's, which writes the output itself; rows without blocks among them."""
    c = Cache(2, (1, 0), 8, [300, 1000, 40, 0] * 40, seed=4)
    import bit_quantized_kv_decode_gb300 as kvq
    assert kvq.sparse_workspace_size(c.desc, 160, 32, 2) == 0
    q = c.queries(4)
    lists = some_lists(c, 2, 5)
    assert_sparse_close(*call(c, q, lists, 2), *attend_lists64(c, q, lists))


def test_long_lists_of_one_sequence():
    """More ranges than one step of the merge takes, and lists longer than what a CTA looks ahead."""
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(2, (1, 0), 1, [128 * 700 - 5], 64, 64, seed=5)
    q = c.queries(8)
    for n in (699, 257, 33):
        lists = [[sorted(random.Random(n).sample(range(700), n))]]
        assert_sparse_close(*call(c, q, lists, 700), *attend_lists64(c, q, lists))
    many = Cache(2, (1, 0), 8, [128 * 90] * 20 + [50] * 140, 64, 32, seed=6)  # ranges of more than 32 blocks
    q = many.queries(1)
    lists = [[list(range(90 if n > 50 else 1)) for _ in range(8)] for n in many.lengths]
    assert_sparse_close(*call(many, q, lists, 90), *attend_lists64(many, q, lists))


def test_whole_lists_equal_decode():
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, (1, 0), 2, [2000, 1500, 100], seed=6)
    q = c.queries(4)
    lists = [[list(range((n + 127) // 128))] * 2 for n in c.lengths]
    out, lse = call(c, q, lists, 16)
    want, want_lse = kvq.decode_attn(c.desc, q, c.k, c.v, c.lens, c.table)
    rms = want.square().mean().sqrt()
    assert ((out.float() - want).abs() <= 2e-2 * rms + 2.0 ** -8 * want.abs()).all()
    assert ((lse - want_lse).abs() <= 1e-2).all()


@pytest.mark.parametrize("repeat", [1, 30])
def test_bad_entries_counts_and_lengths(repeat):
    """Reported; a bad entry has no tokens, a bad count or length no entries (with one range per list, and with
    several)."""
    import bit_quantized_kv_decode_gb300 as kvq
    lens = [2000, 1500, 700, 1900, 300] * repeat
    c = Cache(4, (1, 0), 8, lens, seed=7)
    q = c.queries(4)
    good = [[[0, 3, 5]] * 8, [[2, 11]] * 8, [[1]] * 8, [[4, 14]] * 8, [[0, 2]] * 8] * repeat
    ref, ref_lse = attend_lists64(c, q, good)
    blocks, counts = as_lists(good, 6, 8)

    def run(blocks, counts, expect, changed, table=None):
        """`changed`: {sequence mod 5: lists}."""
        c.status.zero_()
        out, lse = kvq.sparse_decode_attn(c.desc, q, c.k, c.v, c.lens, blocks, counts, c.table if table is None else table,
                                          return_lse=True, dev_status=c.status)
        assert int(c.status.item()) == expect
        want, want_lse = ref.clone(), ref_lse.clone()
        if changed:
            lists = [changed.get(i % 5, x) for i, x in enumerate(good)]
            want, want_lse = attend_lists64(c, q, lists)
        assert_sparse_close(out, lse, want, want_lse)

    run(blocks, counts, 0, {})
    bad = blocks.clone()
    bad[0::5, :, 0], bad[1::5, :, 1] = -1, 12  # (sequence 1 has 12 blocks: 0 ... 11)
    bad[2::5, :, 0] = 2 ** 31 - 1
    run(bad, counts, kvq.DEV_BAD_PAGE, {0: [[3, 5]] * 8, 1: [[2]] * 8, 2: [[]] * 8})
    n = counts.clone()
    n[0::5], n[3::5] = -1, 7
    run(blocks, n, kvq.DEV_BAD_SEQ_LEN, {0: [[]] * 8, 3: [[]] * 8})
    table = c.table.clone()
    table[0::5, 3], table[4::5] = c.pages, -1
    run(blocks, counts, kvq.DEV_BAD_PAGE, {0: [[0, 5]] * 8, 4: [[]] * 8}, table)
    c.lens[1::5] = c.wide * 128 + 1
    run(blocks, counts, kvq.DEV_BAD_SEQ_LEN, {1: [[]] * 8})


@pytest.mark.parametrize("flag", ["FLAG_TEST_STALL", "FLAG_TEST_STALL_MMA"])
@pytest.mark.parametrize("schemes", [(1, 0), (0, 1)])
def test_a_wait_that_runs_out(flag, schemes):
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, schemes, 2, [2000, 1500], seed=8)
    q = c.queries(4)
    lists = [[[0, 3, 5]] * 2, [[2, 11]] * 2]
    call(c, q, lists, 4, expect=kvq.DEV_TIMEOUT, flags=getattr(kvq, flag))
    c.status.zero_()
    assert_sparse_close(*call(c, q, lists, 4), *attend_lists64(c, q, lists))


def test_given_buffers_streams_and_graphs():
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, (1, 0), 2, [2000, 1500, 700], seed=9)
    q = c.queries(4)
    lists = [[[0, 3, 5], [1]], [[2, 11], [4, 5, 6]], [[1], [5]]]
    out, lse = call(c, q, lists, 4)
    memory = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    size = kvq.sparse_workspace_size(c.desc, 3, 8, 4)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    again, _ = call(c, q, lists, 4, out=memory[:3], workspace=ws)
    assert torch.equal(again, out) and (memory[3] == 7).all() and (ws[size:] == 0xFF).all()
    with pytest.raises(kvq.KvqError, match="workspace"):
        call(c, q, lists, 4, workspace=ws[:size - 1])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        other, _ = call(c, q, lists, 4)
    stream.synchronize()
    assert torch.equal(other, out)
    blocks, counts = as_lists(lists, 4, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, got_lse = kvq.sparse_decode_attn(c.desc, q, c.k, c.v, c.lens, blocks, counts, c.table, return_lse=True)
    blocks[0, 1, 0] = 9
    counts[2, 0] = 0
    graph.replay()
    lists[0][1], lists[2][0] = [9], []
    assert_sparse_close(got, got_lse, *attend_lists64(c, q, lists))

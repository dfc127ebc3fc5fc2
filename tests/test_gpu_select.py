"""Selection of blocks against its definition in 64 bits: lists are equal, entry
by entry, ties at the lowest index."""
import numpy as np
import pytest
import torch

from tests.sparse_testlib import Cache, scores64, select64

pytestmark = pytest.mark.gpu


def check(cache, q, budget, first=1, last=1, expect=0, **kw):
    import bit_quantized_kv_decode_gb300 as kvq
    blocks, counts = kvq.select_blocks(cache.desc, q, cache.k, cache.lens, budget, first=first, last=last,
                                       page_table=cache.table, max_blocks=cache.wide, dev_status=cache.status, **kw)
    assert int(cache.status.item()) == expect
    score = scores64(cache, q)
    for b in range(len(cache.lengths)):
        for h in range(cache.hkv):
            want = select64(score[b][h], budget, first, last)
            n = int(counts[b, h])
            assert n == len(want) and blocks[b, h, :n].tolist() == want, (b, h)
            assert (blocks[b, h, n:] == -1).all()
    return blocks, counts


LENS = [1, 128, 129, 2047, 2048, 2049, 3000, 5000, 777, 4097]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("per", [1, 4, 8])
def test_geometries(bits, dim, group, per):
    c = Cache(bits, (1, 0), 2, LENS, dim, group, seed=bits + dim + group + per)
    check(c, c.queries(per), 9)


@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1), (3, 0, 0), (8, 3, 4), (16, 16, 0),
                                               (16, 0, 16), (17, 0, 1), (33, 2, 2), (64, 1, 1), (200, 1, 1)])
def test_budgets(budget, first, last):
    c = Cache(4, (1, 1), 3, LENS, paged=False, seed=budget)
    check(c, c.queries(2), budget, first, last)


def test_long_sequences_over_clusters():
    """Few lists: several CTAs score one; 2,000 blocks are more than a round of any loop."""
    c = Cache(2, (1, 0), 1, [256_000, 100_001], 64, 64, seed=3)
    q = c.queries(4)
    for budget in (5, 700, 1999):
        check(c, q, budget, 1, 3)


def test_equal_blocks_go_by_index():
    """Every block of a sequence on the same page's values: equal scores, exactly."""
    c = Cache(4, (1, 0), 2, [128 * 40, 128 * 300 + 5], seed=4)
    for t in c.k:
        for b, n in enumerate(c.lengths):
            for j in range(1, n // 128):
                t[c.page(b, j)] = t[c.page(b, 0)]
    check(c, c.queries(4), 12)
    c.k[1].zero_(), c.k[2].zero_()  # scores of zero
    check(c, c.queries(4), 12)


def test_zero_queries_and_both_zeros():
    c = Cache(4, (1, 0), 2, [128 * 40], seed=5)
    check(c, torch.zeros_like(c.queries(4)), 7)
    check(c, -torch.zeros_like(c.queries(4)), 7)


@pytest.mark.parametrize("step", [0, 1, 3])
def test_neighbours_that_fp32_cannot_tell_apart(step):
    """Blocks whose scores are sums of large terms that cancel but for the last bit of one offset: differences far below
    an fp32 rounding of the terms decide."""
    c = Cache(4, (1, 0), 1, [128 * 64], seed=6)
    g = torch.Generator().manual_seed(step)
    s, z = torch.zeros_like(c.k[1]), torch.zeros_like(c.k[2])
    big = torch.randn(128, generator=g).half() * 1000
    z[:, 0] = big.cuda()
    for j in range(64):
        z[c.page(0, j), 0, 5] = 2.0 ** -10 * (1 + ((j * 29) % 64) * step / 1024)
    c.k[1].copy_(s), c.k[2].copy_(z)
    check(c, c.queries(4), 20)


def test_large_and_not_finite_queries():
    c = Cache(4, (1, 0), 2, [128 * 40, 128 * 50], seed=7)
    q = c.queries(4)
    check(c, q * 2.0 ** 100, 9)  # fp32 sums overflow, those in 64 bits do not
    check(c, (q * 2.0 ** -130).to(torch.bfloat16), 9)
    bad = q.clone()
    bad[0, 0, 3] = float("nan")
    bad[1, 5, 100] = float("inf")
    check(c, bad, 9)


@pytest.mark.parametrize("small", [-100, -115, -128])
def test_products_that_fp32_does_not_hold(small):
    """Queries times scales and offsets of 2^-20: below 2^-149 in part, or altogether."""
    c = Cache(4, (1, 0), 2, [128 * 40, 128 * 50], seed=11)
    for t in c.k[1:]:
        t.copy_((t.float() * 2.0 ** -20).half())
    q = (c.queries(4).float() * 2.0 ** small).to(torch.bfloat16)
    assert q.any()
    check(c, q, 9)


def test_bad_lengths_and_pages():
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, (1, 0), 2, [128 * 40, 128 * 30, 128 * 20], seed=8)
    q = c.queries(4)
    want, _ = check(c, q, 9)
    for bad in (-1, c.wide * 128 + 1):
        c.lens[1] = bad
        c.status.zero_()
        blocks, counts = kvq.select_blocks(c.desc, q, c.k, c.lens, 9, page_table=c.table, dev_status=c.status)
        assert int(c.status.item()) == kvq.DEV_BAD_SEQ_LEN
        assert (blocks[1] == -1).all() and (counts[1] == 0).all()
        assert torch.equal(blocks[[0, 2]], want[[0, 2]])
    c.lens[1] = 128 * 30
    c.status.zero_()
    c.table[0, 5:30] = c.pages
    c.table[0, 30] = -1
    blocks, counts = kvq.select_blocks(c.desc, q, c.k, c.lens, 20, page_table=c.table, dev_status=c.status)
    assert int(c.status.item()) == kvq.DEV_BAD_PAGE
    # 38 are scored, 26 of them minus infinity: 12 good ones, then the lowest bad ones
    assert blocks[0, 0].tolist() == list(range(11)) + list(range(31, 40))


def test_largest_sequence():
    """16,384 blocks (two million tokens), the most that a selection takes: scales and offsets alone."""
    import bit_quantized_kv_decode_gb300 as kvq
    n = 16384
    desc = kvq.cache_desc(2, 1, 0, 1, n, head_dim=64, group=64)
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(n, 1, 128, generator=g, device="cuda").half()
    s = torch.rand(n, 1, 128, generator=g, device="cuda").half()
    codes = torch.empty(n, 1, kvq.block_bytes(2, 64), dtype=torch.uint8, device="cuda")
    q = torch.randn(1, 8, 64, generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([n * 128 - 70], dtype=torch.int32, device="cuda")
    x = q[0].double()
    score = (z.double().view(n, 2, 64) * x.sum(0)).sum(-1) + 3 * (s.double().view(n, 2, 64) * x.clamp(min=0).sum(0)).sum(-1)
    score[-1, 1] = -np.inf
    score = score.amax(1).cpu().numpy()
    for budget in (1, 64, 5000, n - 1, n):
        blocks, counts = kvq.select_blocks(desc, q, (codes, s, z), lens, budget, first=0, last=1, max_blocks=n)
        want = select64(score, budget, 0, 1)
        assert blocks[0, 0, :len(want)].tolist() == want and int(counts) == len(want)
    flat = torch.zeros_like(z)  # all of them equal
    blocks, _ = kvq.select_blocks(desc, q, (codes, flat + 0.5, flat + 0.25), lens, 100, first=0, last=1, max_blocks=n)
    assert blocks[0, 0].tolist() == list(range(99)) + [n - 1]


def test_given_buffers_streams_and_graphs():
    import bit_quantized_kv_decode_gb300 as kvq
    c = Cache(4, (1, 0), 2, LENS, seed=9)
    q = c.queries(4)
    memory = torch.full((len(LENS) + 1, 2, 9), 77, dtype=torch.int32, device="cuda")
    n = torch.full((len(LENS) + 1, 2), 77, dtype=torch.int32, device="cuda")
    check(c, q, 9, blocks=memory[:-1], counts=n[:-1])
    assert (memory[-1] == 77).all() and (n[-1] == 77).all()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        blocks, _ = kvq.select_blocks(c.desc, q, c.k, c.lens, 9, page_table=c.table)
    stream.synchronize()
    assert torch.equal(blocks, memory[:-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blocks, counts = kvq.select_blocks(c.desc, q, c.k, c.lens, 9, page_table=c.table)
    q.copy_(-q)
    c.lens[3] = c.lengths[3] = 1500
    graph.replay()
    want, _ = check(c, q, 9)
    assert torch.equal(blocks, want)

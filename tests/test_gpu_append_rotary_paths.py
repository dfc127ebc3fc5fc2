"""Append with the position rotation where an ordinary model takes it: many query
heads beside the keys' rows, prompts so long that a CTA takes two columns of a
block, and bad pages and refused sequences among whole blocks."""
import pytest
import torch

from tests.rows_testlib import DTYPES
from tests.test_gpu_append_rotary import Setup, turn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,hkv,heads", [(64, 4, 36), (64, 8, 64), (64, 1, 33), (128, 8, 32), (128, 4, 20), (128, 1, 17),
                                           (256, 8, 32), (256, 4, 20), (256, 9, 9), (128, 40, 40)])
@pytest.mark.parametrize("dtype,interleaved", [("bf16", False), ("fp16", True), ("fp32", False)])
def test_rows_in_several_pieces(dim, hkv, heads, dtype, interleaved):
    """A warp takes 32, 16 or 8 heads (of 64, 128, 256): more pieces than one of q's, of k's, the last one partly full."""
    s = Setup(4, (1, 0), dim, 64, hkv, DTYPES[dtype], dim - 16, interleaved, per=heads // hkv, seed=heads, old=[3, 0, 130],
              new=[70, 0, 41])
    got = s.copies()
    k_out = torch.full_like(s.k, 9.0)
    q = s.rotary(*got, q=s.q, k_out=k_out)
    assert q.shape[1] == heads
    s.check_rows(q, s.q, "q")
    s.check_rows(k_out, s.k, "k")
    s.check_equal(got, s.reference())


@pytest.mark.parametrize("beside", [False, True])  # rows turned beside the blocks
@pytest.mark.parametrize("dim,group,hkv", [(128, 128, 8), (128, 64, 7), (128, 32, 7), (64, 64, 13), (64, 32, 13), (64, 32, 15),
                                           (256, 128, 4), (256, 32, 4)])
@pytest.mark.parametrize("schemes,bits,dtype,interleaved", [((1, 0), 4, "bf16", False), ((0, 1), 2, "fp16", True),
                                                            ((1, 1), 2, "bf16", True), ((0, 0), 4, "fp16", False)])
def test_two_columns_of_a_block(dim, group, hkv, schemes, bits, dtype, interleaved, beside):
    """Columns of 128 channels of 1,824 whole blocks or more; odd numbers of columns (7 heads of 128, 13 of 64) and of
    heads (13 and 15 of 64), blocks that chunks go on into."""
    columns = (hkv * dim + 127) // 128
    blocks = -(-1824 // columns) + 8
    new = [128 * (blocks // 2) + 77, 128 * (blocks // 4) - 1, 5, 128 * (blocks // 4)]
    while sum(new) // 128 * columns < 1824:
        new[0] += 128
    s = Setup(bits, schemes, dim, group, hkv, DTYPES[dtype], dim - 32, interleaved, per=1, seed=dim + hkv, old=[0, 100, 128, 1],
              new=new)
    got = s.copies()
    kw = dict(q=s.q, k_out=torch.full_like(s.k, 9.0)) if beside else {}
    q = s.rotary(*got, **kw)
    want = s.reference()
    s.check_equal(got, want)
    if beside:
        at = slice(sum(new) - 300, None)  # (all rows take the same way)
        s.position, s.q, s.k = s.position[at], s.q[at], s.k[at]
        s.check_rows(q[at], s.q, "q")
        s.check_rows(kw["k_out"][at], s.k, "k")


@pytest.mark.parametrize("what", ["page", "refused", "both"])
@pytest.mark.parametrize("schemes,dim", [((1, 0), 128), ((0, 1), 64), ((1, 1), 256)])
def test_whole_blocks_beside_what_is_skipped(what, schemes, dim):
    """A bad page in the middle of a sequence, a refused sequence between good ones: reported, that block and that
    sequence (its windows too) left as they were, everything else written.  A sequence's window holds its new rows
    although the page of their block is bad."""
    base = dict(old=[10, 20, 30, 0], new=[600, 700, 500, 650], seed=9)
    s = Setup(4, schemes, dim, 64, 2, torch.bfloat16, dim, **base)
    assert sum(s.new) >= 64 * len(s.new)  # (kernels for whole blocks)
    want = s.reference()
    pages = s.page_table.clone().cpu()
    got, skipped, expect = s.copies(), [], 0
    if what != "refused":  # whole blocks, a first and a last one
        for b, j in (0, 2), (2, 1), (3, 0), (3, 5):
            s.page_table[b, j] = s.desc.num_pages + b
            skipped.append(int(pages[b, j]))
        expect |= s.kvq.DEV_BAD_PAGE
    if what != "page":
        s.lens[1] = -1
        skipped += [int(p) for p in pages[1, :6]]
        expect |= s.kvq.DEV_BAD_SEQ_LEN
    q_out, k_out = torch.full_like(s.q, 7.0), torch.full_like(s.k, 7.0)
    s.rotary(*got, q=s.q, q_out=q_out, k_out=k_out)
    assert int(s.status.item()) == expect
    good = [int(p) for b, n in enumerate(s.total) for p in pages[b, :(n + 127) // 128] if int(p) not in skipped]
    for c, was, w in zip(got[0], s.cache, want[0]):
        for a, b, d in zip(c, was, w):
            assert torch.equal(a[skipped].view(torch.uint8), b[skipped].view(torch.uint8))
            assert torch.equal(a[good].view(torch.uint8), d[good].view(torch.uint8))
    refused = [1] if what != "page" else []
    for a, was, w in zip(got[1], s.window, want[1]):
        for b in range(4):
            assert torch.equal(a[b], (was if b in refused else w)[b])
    rows = torch.zeros(len(s.q), dtype=torch.bool, device="cuda")
    rows[600:1300] = what != "page"
    assert (q_out[rows] == 7).all() and (k_out[rows] == 7).all()
    s.position = s.position[~rows]
    s.check_rows(q_out[~rows], s.q[~rows], "q")
    s.check_rows(k_out[~rows], s.k[~rows], "k")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_without_a_sequence(dtype):
    """Rows in front of the first sequence and behind the last one: a given q_out and k_out keep them."""
    s = Setup(4, (1, 0), 128, 64, 2, DTYPES[dtype], 128, old=[3, 0, 200], new=[4, 130, 9], seed=11)
    want = s.reference()
    got = s.copies()
    T, before, behind = len(s.q), 5, 70

    def padded(x):
        return torch.cat([torch.full_like(x[:1], float("nan")).expand(before, -1, -1), x,
                          torch.full_like(x[:1], float("nan")).expand(behind, -1, -1)])

    q, s.q = s.q, padded(s.q)
    k, s.k, s.v = s.k, padded(s.k), padded(s.v)
    s.cu = s.cu + before
    q_out, k_out = torch.full_like(s.q, 7.0), torch.full_like(s.k, 7.0)
    assert s.rotary(*got, q=s.q, q_out=q_out, k_out=k_out) is q_out
    s.check_equal(got, want)
    at = slice(before, before + T)
    s.check_rows(q_out[at], q, "q")
    s.check_rows(k_out[at], k, "k")
    for x in (q_out, k_out):
        assert (x[:before] == 7).all() and (x[before + T:] == 7).all()


@pytest.mark.parametrize("T", [100, 5000])
def test_rows_that_sequences_share(T):
    """Behind a decreasing entry: reported, and a row is turned for one of its sequences, or left."""
    import bit_quantized_kv_decode_gb300 as kvq
    wide, B, dim = (T + 127) // 128 + 2, 5, 128
    desc = kvq.cache_desc(4, 0, 0, 2, B * wide)
    g = torch.Generator(device="cuda").manual_seed(42)
    q, k, v = (torch.randn(T + 9, h, dim, generator=g, device="cuda") for h in (8, 2, 2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = [0, 3, 50, 3, 90]
    table = kvq.rotary_table(T + 90, dim)
    out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    kvq.append_rotary(desc, table, k, v, torch.tensor([0, T] * 3, dtype=torch.int32, device="cuda"),
                      torch.tensor(old, dtype=torch.int32, device="cuda"), *(kvq.alloc_cache(desc) for _ in "kv"),
                      max_blocks=wide, q=q, q_out=out, k_out=k_out, dev_status=status)
    assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN
    for x, got in ((q, out), (k, k_out)):
        right = (got == 7.0).flatten(1).all(1)
        for b in (0, 2, 4):
            right[:T] |= (got[:T] == turn(x[:T], table[old[b]:old[b] + T], False)).flatten(1).all(1)
        assert right.all() and (got[T:] == 7.0).all()

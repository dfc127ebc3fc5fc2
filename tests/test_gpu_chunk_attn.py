"""Attention of chunks of new tokens over the packed cache against the
definition in 64 bits: every geometry, scheme and width, chunk lengths from
none to several row tiles, caches of one token to many blocks (cut into ranges
and joined), empty rows, bad pages and lengths, streams and graphs."""
import math

import pytest
import torch

import kvq_synth as synth
from tests.rows_testlib import (DTYPES, HALF_STEP, assert_lse_close, assert_rows_close, attend64, cache_values, starts)

pytestmark = pytest.mark.gpu


class Setup:
    def __init__(self, bits=4, schemes=(1, 0), dim=128, group=128, hkv=2, per=4, dtype=torch.bfloat16, paged=True,
                 new=(4, 1), total=(200, 77), seed=1, loud=1.0):
        import bit_quantized_kv_decode_gb300 as kvq
        self.new, self.total, self.schemes, self.bits = list(new), list(total), schemes, bits
        B, L = len(new), max(1, max(total))
        self.wide = max(1, (L + 127) // 128)
        lens = torch.tensor(self.total, dtype=torch.int32)
        if paged:
            self.table, pages = synth.page_table_for(lens, seed, self.wide)
            self.table_dev = self.table.cuda()
        else:
            self.table, self.table_dev, pages = None, None, B * self.wide
        self.desc = kvq.cache_desc(bits, *schemes, hkv, max(1, pages), head_dim=dim, group=group)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens = lens.cuda()
        self.cache = []
        for which in (0, 1):
            x = torch.randn(B, hkv, L, dim, generator=g, device="cuda")
            if which == 0:
                x *= 1 + (loud - 1) * torch.rand(hkv, 1, dim, generator=g, device="cuda")
            cache = kvq.alloc_cache(self.desc)
            for t in cache:  # what unused pages hold must not matter
                t.view(torch.uint8).fill_(0x7E)
            kvq.pack(self.desc, which, x, self.lens, self.table_dev, self.wide, cache=cache)
            self.cache.append(cache)
        self.q = torch.randn(sum(new), hkv * per, dim, generator=g, device="cuda").to(dtype)
        self.cu = starts(new).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        import bit_quantized_kv_decode_gb300 as kvq
        args = dict(max_blocks=self.wide, dev_status=self.status, return_lse=True)
        args.update(kw)
        r = kvq.chunk_attn(self.desc, self.q, *self.cache, self.cu, self.lens, self.table_dev, **args)
        torch.cuda.synchronize()
        return r

    def check(self, got=None, causal=True, sm_scale=0.0, only=None, **kw):
        out, lse = got or self.call(causal=causal, sm_scale=sm_scale, **kw)
        assert int(self.status.item()) == 0
        D = self.q.shape[2]
        scale = sm_scale if sm_scale > 0 else 1.0 / math.sqrt(D)
        k, v = (cache_values([t.cpu() for t in self.cache[w]], self.total, self.bits, w, self.schemes[w], self.table, D)
                for w in (0, 1))
        cu = self.cu.tolist()
        for b, (n, L) in enumerate(zip(self.new, self.total)):
            if only is not None and b not in only:
                continue
            rows = slice(cu[b], cu[b] + n)
            ref, rl, tol, ltol = attend64(self.q[rows], k[b, :L].cuda(), v[b, :L].cuda(), L - n, causal, scale,
                                          HALF_STEP[torch.float16])
            assert_rows_close(out[rows], ref, tol, self.q.dtype, f"sequence {b}: {n} rows, {L} tokens")
            assert_lse_close(lse[rows], rl, ltol, f"sequence {b}")
        return out, lse


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("schemes", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64),
                                       (256, 128)])
def test_geometries(bits, schemes, dim, group):
    s = Setup(bits, schemes, dim, group, new=(4, 1, 0, 33, 130), total=(200, 77, 5, 33, 400), seed=bits + dim + group)
    s.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,total", [((1,), (1,)), ((1, 0, 2), (128, 0, 129)), ((127, 128, 129), (300, 128, 257)),
                                       ((600,), (1000,)), ((0, 0), (0, 7))])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(dim, dtype, new, total, causal):
    s = Setup(dim=dim, group=64, dtype=DTYPES[dtype], new=new, total=total, seed=3)
    s.check(causal=causal)


@pytest.mark.parametrize("hkv,per", [(1, 1), (3, 2), (2, 3), (1, 5), (1, 7), (2, 8), (1, 11), (1, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_head_layouts(hkv, per, dim):
    s = Setup(2, (1, 1), dim, 32, hkv, per, new=(3, 50, 1), total=(130, 260, 1), seed=4)
    s.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,total", [((1, 1, 1), (9000, 130, 4097)), ((5, 17), (20000, 3)), ((300,), (6000,)),
                                       ((32, 32, 32, 31), (640, 8192, 1000, 2561))])
@pytest.mark.parametrize("paged", [False, True])
def test_long_caches_are_cut_and_joined(dim, new, total, paged):
    s = Setup(4, (1, 0), dim, 64, 2, 4, new=new, total=total, paged=paged, seed=5)
    s.check()


def test_loud_channels_and_scale():
    s = Setup(4, (1, 0), 128, 128, 1, 8, new=(40,), total=(3000,), seed=6, loud=40.0)
    s.check()
    s.check(sm_scale=1.0)
    s.check(sm_scale=1e-4, causal=False)


@pytest.mark.parametrize("exponent", [-130, -60, -14, 14, 60])
def test_query_magnitudes(exponent):
    """bf16 queries far outside the fp16 range, the rows of very different size."""
    s = Setup(2, (0, 0), 128, 128, 1, 4, new=(70,), total=(500,), seed=7)
    f = torch.exp2(torch.linspace(0, exponent, 70, device="cuda").round())
    s.q = (s.q.float() * f[:, None, None]).to(torch.bfloat16)
    s.check(sm_scale=2.0 ** -max(0, exponent - 3))


@pytest.mark.parametrize("exponent", [-130, -14, 60])
@pytest.mark.parametrize("dim,n", [(128, 9), (64, 20), (256, 40)])
def test_query_magnitudes_of_few_rows(exponent, dim, n):
    s = Setup(4, (1, 0), dim, 64, 1, 3, new=(n,), total=(500,), seed=18)
    f = torch.exp2(torch.linspace(0, exponent, n, device="cuda").round())
    s.q = (s.q.float() * f[:, None, None]).to(torch.bfloat16)
    s.check(sm_scale=2.0 ** -max(0, exponent - 3))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [(6, 3), (70, 90)])
def test_queries_that_are_not_finite_stay_in_their_rows(dtype, new):
    s = Setup(dtype=DTYPES[dtype], new=new, total=(500, 1400), seed=19)
    good, good_lse = s.check()
    s.q[2, 1, 5] = math.nan
    s.q[4, 0, 7] = math.inf
    out, lse = s.call()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])
    assert out[2, 1].isnan().all() and lse[2, 1].isnan()


def test_rows_before_the_first_token_are_empty():
    """Chunks longer than what the cache holds: rows at negative positions."""
    s = Setup(new=(10, 200), total=(4, 130), seed=8)
    out, lse = s.check()
    assert (out[:6] == 0).all() and (lse[:6] == -math.inf).all()
    assert (out[10:80] == 0).all() and (lse[10:80] == -math.inf).all()


def test_rows_outside_every_sequence():
    s = Setup(new=(50, 3), total=(300, 40), seed=9)
    q = torch.full((90, *s.q.shape[1:]), math.nan, dtype=s.q.dtype, device="cuda")
    q[17:70] = s.q
    s.q, s.cu = q, s.cu + 17
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    s.check(out=out, lse=lse)
    for x in (out, lse):
        assert (x[:17] == 7).all() and (x[70:] == 7).all()


def test_strided_queries():
    s = Setup(new=(50, 3), total=(300, 40), seed=10)
    wide = torch.randn(53, 3 * s.q.shape[1], 128, device="cuda").to(s.q.dtype)
    wide[:, 8:16] = s.q
    s.q = wide[:, 8:16]
    s.check()


def test_single_tokens_agree_with_decode():
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(4, (1, 0), 128, 128, 2, 4, new=(1, 1, 1), total=(700, 128, 1), seed=11)
    out, lse = s.check()
    o, l = kvq.decode_attn(s.desc, s.q, *s.cache, s.lens, s.table_dev, mode=kvq.OPERANDS_BF16)
    rms = o.double().pow(2).mean().sqrt()
    assert (out.double() - o.double()).abs().max() <= 2.0 ** -6 * rms * 3
    assert (lse - l).abs().max() <= 2e-3 + 2.0 ** -8


@pytest.mark.parametrize("paged", [False, True])
def test_bad_lengths_and_pages_are_flagged(paged):
    import bit_quantized_kv_decode_gb300 as kvq
    for what in ("long", "negative", "page", "starts"):
        s = Setup(new=(20, 30, 10), total=(300, 280, 290), seed=12, paged=paged)
        good, good_lse = s.check()
        s.status.zero_()
        if what == "long":
            s.lens[1] = s.wide * 128 + 1
        elif what == "negative":
            s.lens[1] = -5
        elif what == "page":
            if not paged:
                continue
            s.table_dev[1, 1] = s.desc.num_pages
        else:
            s.cu[1:3] = torch.tensor([30, 20])
        out, lse = s.call()
        assert int(s.status.item()) == (kvq.DEV_BAD_PAGE if what == "page" else kvq.DEV_BAD_SEQ_LEN)
        if what == "starts":
            continue
        assert torch.equal(out[:20], good[:20]) and torch.equal(out[50:], good[50:])
        assert torch.isfinite(out).all()
        if what != "page":
            assert (out[20:50] == 0).all() and (lse[20:50] == -math.inf).all()


@pytest.mark.parametrize("schemes", [(0, 0), (1, 1)])
def test_values_past_the_fp16_range(schemes):
    """A group whose values do not fit fp16: reported, lowered to fit."""
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(4, schemes, 128, 128, 1, 2, new=(3,), total=(140,), seed=13)
    for w in (0, 1):
        s.cache[w][1][:, :, 5] = 60000.0
        s.cache[w][2][:, :, 5] = 100.0
    out, lse = s.call()
    assert int(s.status.item()) == kvq.DEV_NONFINITE
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and out.abs().max() <= 65504


def test_repeatable_with_and_without_workspace():
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(2, (1, 0), 128, 128, 2, 4, new=(5, 9, 1), total=(9000, 100, 5000), seed=14)
    a, la = s.call()
    n = kvq.chunk_workspace_size(s.desc, 3, 15, 8, s.wide)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        b, lb = s.call(workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    with pytest.raises(kvq.KvqError):
        s.call(workspace=ws[:-1])


def test_streams_and_graphs():
    """Two calls on two streams at once, and a captured call replayed on other
    lengths and queries."""
    import bit_quantized_kv_decode_gb300 as kvq
    sets = [Setup(4, (1, 0), 128, 128, 2, 4, new=n, total=t, seed=15) for n, t in
            (((5, 9), (4000, 3900)), ((13, 1), (130, 4000)))]
    want = [s.call()[0] for s in sets]
    side = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (s, st) in enumerate(zip(sets, side)):
            with torch.cuda.stream(st):
                got[i] = kvq.chunk_attn(s.desc, s.q, *s.cache, s.cu, s.lens, s.table_dev)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = sets[0]
    q, cu, lens = s.q.clone(), s.cu.clone(), s.lens.clone()
    ws = torch.empty(kvq.chunk_workspace_size(s.desc, 2, 14, 8, s.wide), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.chunk_attn(s.desc, q, *s.cache, cu, lens, s.table_dev, out=out, workspace=ws)
    new = torch.tensor([0, 2, 14], dtype=torch.int32)
    s.cu, s.new, s.total = new.cuda(), [2, 12], [1000, 2049]
    s.lens = torch.tensor(s.total, dtype=torch.int32, device="cuda")
    other = s.call()[0]
    for c, n, w in ((new, s.lens, other), (starts((5, 9)), torch.tensor((4000, 3900), dtype=torch.int32), want[0])):
        cu.copy_(c)
        lens.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_many_sequences():
    g = torch.Generator().manual_seed(2)
    new = torch.randint(0, 4, (700,), generator=g).tolist()
    total = [n + int(x) for n, x in zip(new, torch.randint(0, 140, (700,), generator=g))]
    s = Setup(2, (0, 1), 64, 64, 1, 4, new=new, total=total, seed=16)
    s.check(only=[0, 1, 31, 32, 33, 64, 500, 698, 699])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [(3, 2), (400, 300)])
def test_withheld_copies_time_out(dim, new):
    """A copy that never arrives ends in a status, not in a hang; the next call
    is right again."""
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(4, (1, 0), dim, 64, 2, 4, new=new, total=(900, 700), seed=17)
    s.call(flags=kvq.FLAG_TEST_STALL)
    assert int(s.status.item()) & kvq.DEV_TIMEOUT
    s.status.zero_()
    s.check()

"""Attention over whole prompts against the definition in 64 bits: head
layouts, lengths from zero and one token to several tiles, strides, types,
values in masked places, rows outside every sequence, streams and graphs."""
import math

import pytest
import torch

from tests.rows_testlib import DTYPES, HALF_STEP, assert_lse_close, assert_rows_close, attend64, starts

pytestmark = pytest.mark.gpu


def make(T, Hq, Hkv, D, dtype, seed, layout="separate", loud=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")
    qkv[:, Hq:Hq + Hkv] *= loud
    qkv = qkv.to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if layout == "separate":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    elif layout == "heads_first":  # [heads, tokens, channels] in memory
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    return q, k, v


def check(q, k, v, lens, causal=True, sm_scale=0.0, first=0, got=None):
    import bit_quantized_kv_decode_gb300 as kvq
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = starts(lens, first).cuda()
    out, lse = got or kvq.prompt_attn(q, k, v, cu, causal=causal, sm_scale=sm_scale, return_lse=True,
                                      dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    scale = sm_scale if sm_scale > 0 else 1.0 / math.sqrt(q.shape[2])
    a = first
    for b, n in enumerate(lens):
        rows = slice(a, a + n)
        a += n
        ref, rl, tol, ltol = attend64(q[rows], k[rows], v[rows], 0, causal, scale, HALF_STEP[q.dtype])
        assert_rows_close(out[rows], ref, tol, q.dtype, f"sequence {b} of {n} tokens")
        assert_lse_close(lse[rows], rl, ltol, f"sequence {b}")
    return out, lse


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 0], [127, 128, 129], [300, 1, 0, 513], [64, 257, 33, 1000]])
def test_lengths(dim, dtype, causal, lens):
    q, k, v = make(sum(lens), 8, 2, dim, DTYPES[dtype], seed=dim + sum(lens))
    check(q, k, v, lens, causal)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hkv,per", [(1, 1), (3, 2), (2, 3), (1, 5), (1, 6), (2, 7), (1, 8), (1, 11), (1, 16)])
def test_head_layouts(dim, hkv, per):
    lens = [259, 40, 131]
    q, k, v = make(sum(lens), hkv * per, hkv, dim, torch.bfloat16, seed=hkv + per)
    check(q, k, v, lens)


@pytest.mark.parametrize("layout", ["fused", "heads_first"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_strided_rows(layout, dim):
    lens = [200, 333]
    q, k, v = make(sum(lens), 8, 4, dim, torch.bfloat16, seed=5, layout=layout)
    assert not q.is_contiguous()
    check(q, k, v, lens)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_prompt_and_loud_channels(dim):
    """Several key tiles per row tile, a peaked softmax whose maximum moves late
    in the row, and an explicit scale."""
    lens = [3001, 517]
    q, k, v = make(sum(lens), 4, 2, dim, torch.bfloat16, seed=9, loud=6.0)
    check(q, k, v, lens)
    k[2900:2910] *= 8  # a late, much larger score: every statistic is rescaled
    check(q, k, v, lens, causal=False)
    check(q, k, v, lens, sm_scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rising_scores(dtype):
    """Scores that rise along the keys (the running maximum moves in every
    tile), and scores so low that plain exponentials would all be zero."""
    T, D = 1200, 128
    q = torch.ones(T, 2, D, device="cuda", dtype=DTYPES[dtype])
    k = (torch.arange(T, device="cuda").float().view(T, 1, 1) / 16).expand(T, 1, D).to(DTYPES[dtype]).contiguous()
    v = torch.randn(T, 1, D, device="cuda").to(DTYPES[dtype])
    check(q, k, v, [T], causal=False, sm_scale=0.05)
    check(q, k - 100, v, [T], causal=True, sm_scale=0.05)
    check(-q, k, v, [T], causal=True, sm_scale=0.05)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_outside_every_sequence(dim, bad):
    """Rows before, between and after the sequences are neither read into a
    result nor written."""
    import bit_quantized_kv_decode_gb300 as kvq
    first, n, T = 37, 150, 400
    q, k, v = make(T, 4, 2, dim, torch.bfloat16, seed=3)
    for x in (q, k, v):
        x[:first] = bad
        x[first + n:] = bad
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, 4), 7.0, device="cuda")
    got = kvq.prompt_attn(q, k, v, starts([n], first).cuda(), out=out, lse=lse)
    check(q, k, v, [n], first=first, got=got)
    for x in (out, lse):
        assert (x[:first] == 7).all() and (x[first + n:] == 7).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 77, 128, 300, 399])
def test_later_tokens_do_not_reach_earlier_rows(dim, bad, at):
    """A token that is not finite changes no row before it, and every row from
    it on, as the formula says."""
    import bit_quantized_kv_decode_gb300 as kvq
    T = 400
    q, k, v = make(T, 4, 1, dim, torch.bfloat16, seed=4)
    cu = starts([T]).cuda()
    clean = kvq.prompt_attn(q, k, v, cu)
    for name in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        (kk if name == "k" else vv)[at, :, 5] = bad
        out = kvq.prompt_attn(q, kk, vv, cu)
        assert torch.equal(out[:at], clean[:at]), name
        if name == "v":
            hit = out[at:, :, 5]
            assert (torch.isnan(hit) if math.isnan(bad) else hit == bad).all()
            assert torch.equal(out[at:, :, :5], clean[at:, :, :5]) and torch.equal(out[at:, :, 6:], clean[at:, :, 6:])


def test_offsets_past_32_bits():
    """Token strides that put the last rows past 2^32 bytes."""
    import bit_quantized_kv_decode_gb300 as kvq
    T, D, st = 1100, 128, 1 << 21
    base = torch.empty(T * st, dtype=torch.bfloat16, device="cuda")
    views = [base.as_strided((T, 2, D), (st, D, 1), i * 1024) for i in range(3)]
    q, k, v = make(T, 2, 2, D, torch.bfloat16, seed=6)
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    check(*views, [T])
    del base, views
    torch.cuda.empty_cache()


def test_bad_starts_are_flagged():
    """A decreasing or out-of-range entry empties its sequence and is reported;
    the others come out right."""
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(300, 4, 2, 128, torch.bfloat16, seed=8)
    for cu, good in (([0, 100, 80, 200], [(0, 100), (80, 200)]), ([0, 50, 301], [(0, 50)]), ([-1, 50, 300], [(50, 300)])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 7.0)
        kvq.prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out, dev_status=status)
        assert int(status.item()) == kvq.DEV_BAD_SEQ_LEN
        for a, e in good:
            alone = kvq.prompt_attn(q[a:e], k[a:e], v[a:e], starts([e - a]).cuda())
            own = [r for r in range(a, e) if cu != [0, 100, 80, 200] or not 80 <= r < 100]  # 80 to 100 belong to two
            assert torch.equal(out[own], alone[[r - a for r in own]])


def test_repeatable_and_without_lse():
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(1500, 8, 2, 128, torch.bfloat16, seed=10)
    cu = starts([700, 800]).cuda()
    a, _ = kvq.prompt_attn(q, k, v, cu, return_lse=True)
    assert torch.equal(a, kvq.prompt_attn(q, k, v, cu))


def test_streams_and_graphs():
    """A call on another stream, and a captured call replayed on new inputs of
    other lengths."""
    import bit_quantized_kv_decode_gb300 as kvq
    T = 600
    sets = [make(T, 8, 2, 128, torch.bfloat16, seed=s) for s in (11, 12)]
    lens = [[300, 300], [1, 512]]
    want = [kvq.prompt_attn(*x, starts(n).cuda()) for x, n in zip(sets, lens)]
    side = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, x, n in zip(side, sets, lens):
        with torch.cuda.stream(s):
            got.append(kvq.prompt_attn(*x, starts(n).cuda()))
    torch.cuda.synchronize()
    for a, b, n in zip(got, want, lens):
        assert torch.equal(a[:sum(n)], b[:sum(n)])
    q, k, v = (x.clone() for x in sets[0])
    cu = starts(lens[0]).cuda()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.prompt_attn(q, k, v, cu, out=out)
    for i in (1, 0):
        for x, y in zip((q, k, v), sets[i]):
            x.copy_(y)
        cu.copy_(starts(lens[i]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:sum(lens[i])], want[i][:sum(lens[i])])


def test_many_sequences():
    """More sequences than one scan of the lengths takes at once, most of them
    of a token or none."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 3, (3000,), generator=g).tolist()
    lens[1234] = 400
    lens[2999] = 129
    q, k, v = make(sum(lens), 2, 1, 64, torch.bfloat16, seed=13)
    import bit_quantized_kv_decode_gb300 as kvq
    out = kvq.prompt_attn(q, k, v, starts(lens).cuda())
    cu = starts(lens).tolist()
    for b in [0, 1, 2, 31, 32, 33, 1233, 1234, 1235, 2998, 2999]:
        if lens[b] == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        ref, _, tol, _ = attend64(q[rows], k[rows], v[rows], 0, True, 1 / 8, HALF_STEP[q.dtype])
        assert_rows_close(out[rows], ref, tol, q.dtype, f"sequence {b}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_withheld_copies_time_out(dim):
    """A copy that never arrives ends in a status, not in a hang; the next call
    is right again."""
    import bit_quantized_kv_decode_gb300 as kvq
    q, k, v = make(700, 4, 2, dim, torch.bfloat16, seed=14)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attn(q, k, v, starts([700]).cuda(), dev_status=status, flags=kvq.FLAG_TEST_STALL)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.DEV_TIMEOUT
    check(q, k, v, [700])

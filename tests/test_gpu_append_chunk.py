"""Appending chunks: the packed bytes equal the oracle's pack of the whole
sequence for every geometry, scheme, type and cache layout, whatever the
chunk's place in its blocks; the windows; calls that are repeated, refused or
captured."""
import numpy as np
import pytest
import torch

import kvq_synth as synth
from oracle import kvq_oracle as orc
from tests.rows_testlib import DTYPES, starts

pytestmark = pytest.mark.gpu

# tokens cached before -> chunk length: block starts and ends, chunks inside a
# block, across several blocks, of one token and of none
OLD = [0, 0, 128, 100, 100, 127, 300, 5, 50, 0]
NEW = [1, 128, 129, 20, 28, 2, 700, 0, 400, 0]


def windows_of(x, lens, hkv, dim):
    w = torch.zeros(len(lens), hkv, 128, dim, device="cuda")
    for b, n in enumerate(lens):
        if n % 128:
            w[b, :, :n % 128] = x[b][n - n % 128:n].transpose(0, 1)
    return w


class Setup:
    def __init__(self, bits, schemes, dim, group, hkv, dtype, paged, seed, old=OLD, new=NEW):
        import bit_quantized_kv_decode_gb300 as kvq
        self.old, self.new, self.schemes, self.bits, self.group = old, new, schemes, bits, group
        self.total = [a + b for a, b in zip(old, new)]
        B = len(old)
        self.wide = max(1, max((n + 127) // 128 for n in self.total))
        lens = torch.tensor(self.total, dtype=torch.int32)
        if paged:
            self.table, pages = synth.page_table_for(lens, seed, self.wide)
            self.table_dev = self.table.cuda()
        else:
            self.table, self.table_dev, pages = None, None, B * self.wide
        self.pages = max(1, pages)
        self.desc = kvq.cache_desc(bits, *schemes, hkv, self.pages, head_dim=dim, group=group)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.rows, self.cache, self.window = [], [], [], []
        for which in (0, 1):
            xs = [torch.randn(n, hkv, dim, generator=g, device="cuda").to(dtype) for n in self.total]
            self.x.append([t.float() for t in xs])
            self.rows.append(torch.cat([t[o:] for t, o in zip(xs, old)]))
            cache = kvq.alloc_cache(self.desc)
            for t in cache:  # recycled pages: what they hold must not matter
                t.view(torch.uint8).fill_(0xA7)
            most = max(1, max(old))
            pad = torch.zeros(B, hkv, most, dim, device="cuda")
            for b, o in enumerate(old):
                pad[b, :, :o] = self.x[which][b][:o].transpose(0, 1)
            kvq.pack(self.desc, which, pad, torch.tensor(old, dtype=torch.int32, device="cuda"), self.table_dev,
                     self.wide, cache=cache)
            self.cache.append(cache)
            self.window.append(windows_of(self.x[which], old, hkv, dim))
        self.cu, self.lens = starts(new).cuda(), torch.tensor(old, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        import bit_quantized_kv_decode_gb300 as kvq
        args = dict(k_window=self.window[0], v_window=self.window[1], page_table=self.table_dev, max_blocks=self.wide,
                    dev_status=self.status)
        args.update(kw)
        kvq.append_chunk(self.desc, self.rows[0], self.rows[1], self.cu, self.lens, *self.cache, **args)
        torch.cuda.synchronize()

    def check(self, windows=None):
        assert int(self.status.item()) == 0
        pages = sorted(int(self.table[b, j]) if self.table is not None else b * self.wide + j
                       for b, n in enumerate(self.total) for j in range((n + 127) // 128))
        for which in (0, 1):
            hkv, dim = self.x[which][0].shape[1:]
            pad = np.zeros((len(self.total), hkv, self.wide * 128, dim), np.float32)
            for b, n in enumerate(self.total):
                pad[b, :, :n] = self.x[which][b].transpose(0, 1).cpu().numpy()
            ref = orc.pack_cache(pad, self.total, self.bits, self.schemes[which], which,
                                 None if self.table is None else self.table.numpy(), self.pages, self.group)
            for name, got, want in zip(("codes", "scale", "zero"), self.cache[which], ref):
                got = got.cpu().view(torch.int16 if name != "codes" else torch.uint8).numpy()
                want = want.view(np.int16) if name != "codes" else want
                assert np.array_equal(got[pages], want[pages]), (name, which)
            if windows is not None:
                want = windows_of(self.x[which], self.total, hkv, dim)
                for b, n in enumerate(self.total):
                    assert torch.equal(windows[which][b, :, :n % 128], want[b, :, :n % 128]), (which, b)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("schemes", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64),
                                       (256, 128)])
def test_equals_pack_of_whole_sequence(bits, schemes, dim, group):
    s = Setup(bits, schemes, dim, group, 2, torch.bfloat16, paged=True, seed=bits + dim + group)
    s.call()
    s.check(s.window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("schemes", [(0, 0), (1, 1)])
def test_types_and_separate_windows(dtype, paged, schemes):
    """window_out apart from the window: the window is left as it was, and the
    call can be made again with the same result."""
    s = Setup(4, schemes, 128, 128, 3, DTYPES[dtype], paged, seed=7)
    before = [w.clone() for w in s.window]
    outs = [torch.full_like(w, 9.0) for w in s.window]
    for _ in range(2):
        s.call(k_window_out=outs[0], v_window_out=outs[1])
        s.check(outs)
    for w, was, o in zip(s.window, before, outs):
        assert torch.equal(w, was)
        for b, n in enumerate(s.total):
            assert (o[b, :, n % 128:] == 9).all()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_token_wise_without_windows(bits, dim, group):
    s = Setup(bits, (0, 0), dim, group, 2, torch.bfloat16, paged=True, seed=3)
    s.call(k_window=None, v_window=None)
    s.check()


def test_strided_rows():
    s = Setup(4, (1, 0), 128, 128, 4, torch.bfloat16, paged=True, seed=5)
    T = s.rows[0].shape[0]
    fused = torch.randn(T, 16, 128, device="cuda").to(torch.bfloat16)
    fused[:, 8:12], fused[:, 12:] = s.rows[0], s.rows[1]
    s.rows = [fused[:, 8:12], fused[:, 12:]]
    s.call()
    s.check(s.window)


def test_then_append_and_chunk_by_chunk():
    """Chunks of several sizes one after another, then single tokens through
    kvq.append with the same windows."""
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(4, (1, 0), 128, 64, 2, torch.bfloat16, paged=True, seed=6, old=[0, 0], new=[500, 391])
    xs = s.x
    cur = [0, 0]
    for step in ([100, 1], [28, 126], [1, 2], [300, 250], [60, 3]):
        rows = [torch.cat([xs[w][b][cur[b]:cur[b] + step[b]] for b in (0, 1)]) for w in (0, 1)]
        kvq.append_chunk(s.desc, *rows, starts(step).cuda(), torch.tensor(cur, dtype=torch.int32, device="cuda"),
                         *s.cache, *s.window, page_table=s.table_dev, dev_status=s.status)
        cur = [a + b for a, b in zip(cur, step)]
    lens = torch.tensor(cur, dtype=torch.int32, device="cuda")
    while cur[0] < 500 or cur[1] < 391:
        assert cur[0] < 500 and cur[1] < 391
        for w in (0, 1):
            x = torch.stack([xs[w][b][cur[b]] for b in (0, 1)])
            kvq.append(s.desc, w, x, lens, s.cache[w], s.window[w], page_table=s.table_dev, dev_status=s.status)
        lens += 1
        cur = [c + 1 for c in cur]
        if cur[0] == 500 or cur[1] == 391:
            break
    s.total = cur
    s.x = [[t[:c] for t, c in zip(xs[w], cur)] for w in (0, 1)]
    s.check(s.window)


@pytest.mark.parametrize("schemes", [(0, 0), (1, 1)])
def test_values_that_are_refused(schemes):
    """NaN and infinity leave their group zero and are reported; the rest of the
    chunk is as it would be."""
    import bit_quantized_kv_decode_gb300 as kvq
    s = Setup(4, schemes, 128, 64, 1, torch.bfloat16, paged=False, seed=9, old=[0], new=[200])
    s.call()
    s.check(s.window)
    want = [kvq.dequant(s.desc, w, s.cache[w], 1, 200, max_blocks=s.wide) for w in (0, 1)]
    for bad in (float("nan"), float("inf"), -float("inf")):
        rows = [r.clone() for r in s.rows]
        rows[0][70, 0, 3] = bad
        s.status.zero_()
        kvq.append_chunk(s.desc, rows[0], rows[1], s.cu, s.lens, *s.cache, *s.window, max_blocks=s.wide,
                         dev_status=s.status)
        assert int(s.status.item()) == kvq.DEV_NONFINITE
        k, v = (kvq.dequant(s.desc, w, s.cache[w], 1, 200, max_blocks=s.wide) for w in (0, 1))
        assert torch.equal(v, want[1])
        group = torch.zeros_like(k, dtype=torch.bool)
        if schemes[0] == 0:
            group[:, :, 70, :64] = True
        else:
            group[:, :, 64:128, 3] = True
        assert (k[group] == 0).all() and torch.equal(k[~group], want[0][~group])


def test_bad_lengths_and_pages_are_flagged():
    import bit_quantized_kv_decode_gb300 as kvq
    base = dict(old=[10, 20, 30], new=[150, 150, 150])
    s = Setup(4, (0, 1), 128, 128, 2, torch.bfloat16, paged=True, seed=4, **base)
    was = [[t.clone() for t in c] for c in s.cache]
    good = [int(p) for b in (0, 2) for p in s.table[b]]
    s.call()
    s.check(s.window)
    done = [[t.clone() for t in c] for c in s.cache]
    for what in ("long", "negative", "page", "starts"):
        s = Setup(4, (0, 1), 128, 128, 2, torch.bfloat16, paged=True, seed=4, **base)
        if what == "long":
            s.lens[1] = 256 - 149
        elif what == "negative":
            s.lens[1] = -1
        elif what == "page":
            s.table_dev[1] = s.pages
        else:
            s.cu[1:3] = torch.tensor([150, 149])
        s.call()
        assert int(s.status.item()) == (kvq.DEV_BAD_PAGE if what == "page" else kvq.DEV_BAD_SEQ_LEN)
        for c, d, w in zip(s.cache, done, was):
            for got, want, old in zip(c, d, w):
                if what != "starts":
                    assert torch.equal(got[good], want[good])
                bad = [int(p) for p in s.table[1]]
                assert torch.equal(got[bad].view(torch.uint8), old[bad].view(torch.uint8))


def test_captured_call_takes_new_lengths():
    s = Setup(2, (1, 0), 64, 32, 2, torch.float16, paged=True, seed=8)
    cu, lens = s.cu.clone(), s.lens.clone()
    s.cu.zero_()
    graph = torch.cuda.CUDAGraph()
    import bit_quantized_kv_decode_gb300 as kvq
    s.call()
    with torch.cuda.graph(graph):
        kvq.append_chunk(s.desc, s.rows[0], s.rows[1], s.cu, s.lens, *s.cache, *s.window, page_table=s.table_dev,
                         dev_status=s.status)
    s.cu.copy_(cu)
    graph.replay()
    torch.cuda.synchronize()
    s.check(s.window)


def test_nothing_to_append():
    s = Setup(4, (1, 0), 128, 128, 2, torch.bfloat16, paged=True, seed=2, old=[5, 128, 300], new=[0, 0, 0])
    was = [[t.clone() for t in c] for c in s.cache]
    outs = [torch.full_like(w, 9.0) for w in s.window]
    s.call(k_window_out=outs[0], v_window_out=outs[1])
    for c, w in zip(s.cache, was):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c, w))
    s.check(outs)

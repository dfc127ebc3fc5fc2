"""Append with the position rotation: the cache and the windows equal, byte for
byte, what append_chunk makes of fp32 rows turned by single fp32 operations (and
so the oracle's pack of the whole sequence); turned queries and keys against 64
bits; calls that are strided, repeated, captured, refused on the device."""
import numpy as np
import pytest
import torch

import kvq_synth as synth
from oracle import kvq_oracle as orc
from tests.rows_testlib import DTYPES, HALF_STEP, starts

pytestmark = pytest.mark.gpu

OLD = [0, 0, 128, 100, 100, 127, 300, 5, 50, 0]
NEW = [1, 128, 129, 20, 28, 2, 700, 0, 400, 0]


def turn(x, angle, interleaved, dtype=torch.float32):
    """x [T, H, D], angle [T, R]; every operation rounded to `dtype` by itself."""
    x, angle = x.to(dtype), angle.to(dtype)
    R = angle.shape[1]
    c, s = angle[:, None, :R // 2], angle[:, None, R // 2:]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Setup:
    def __init__(self, bits, schemes, dim, group, hkv, dtype, rotary, interleaved=False, paged=True, seed=1, old=OLD, new=NEW,
                 per=2, windows=True):
        import bit_quantized_kv_decode_gb300 as kvq
        self.kvq, self.old, self.new, self.interleaved, self.schemes = kvq, old, new, interleaved, schemes
        self.total = [a + b for a, b in zip(old, new)]
        B, T = len(old), sum(new)
        self.wide = max(1, max((n + 127) // 128 for n in self.total))
        if paged:
            table, pages = synth.page_table_for(torch.tensor(self.total), seed, self.wide)
            self.page_table = table.cuda()
        else:
            self.page_table, pages = None, B * self.wide
        self.desc = kvq.cache_desc(bits, *schemes, hkv, max(1, pages), head_dim=dim, group=group)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = torch.randn(T, per * hkv, dim, generator=g, device="cuda").to(dtype)
        self.k, self.v = (torch.randn(T, hkv, dim, generator=g, device="cuda").to(dtype) for _ in "kv")
        self.table = kvq.rotary_table(max(self.total) + 3, rotary)
        self.cu, self.lens = starts(new).cuda(), torch.tensor(old, dtype=torch.int32, device="cuda")
        self.position = torch.cat([torch.arange(o, o + n) for o, n in zip(old, new)]).cuda()
        self.cache = [self.noise(kvq.alloc_cache(self.desc)) for _ in "kv"]
        self.window = [torch.randn(B, hkv, 128, dim, generator=g, device="cuda") for _ in "kv"] if windows else [None, None]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @staticmethod
    def noise(cache):
        for t in cache:  # what pages hold must not matter (no NaN as a half: 0x2727)
            t.view(torch.uint8).fill_(0x27)
        return cache

    def copies(self):
        return [tuple(t.clone() for t in c) for c in self.cache], [None if w is None else w.clone() for w in self.window]

    def rotary(self, cache, window, **kw):
        args = dict(page_table=self.page_table, max_blocks=self.wide, interleaved=self.interleaved, dev_status=self.status)
        args.update(kw)
        return self.kvq.append_rotary(self.desc, self.table, self.k, self.v, self.cu, self.lens, *cache, *window, **args)

    def reference(self):
        """append_chunk of the turned rows, K and V each from fp32 rows."""
        cache, window = self.copies()
        k = turn(self.k, self.table[self.position], self.interleaved)
        self.kvq.append_chunk(self.desc, k, self.v.float(), self.cu, self.lens, *cache, *window, page_table=self.page_table,
                              max_blocks=self.wide)
        return cache, window

    def check_equal(self, got, want):
        assert int(self.status.item()) == 0
        for c, d in zip(got[0], want[0]):
            for a, b in zip(c, d):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(got[1], want[1]):
            assert a is None and b is None or torch.equal(a, b)

    def check_rows(self, got, x, what):
        """Each of the three operations is off by 2^-24 of its result at most; then one rounding to the type."""
        angle = self.table[self.position]
        ref = turn(x, angle, self.interleaved, torch.float64)
        mag = turn(x.abs().double(), torch.cat([angle[:, :angle.shape[1] // 2].abs(), -angle[:, angle.shape[1] // 2:].abs()], 1),
                   self.interleaved, torch.float64)
        mag = torch.maximum(mag, x.abs().double())  # |x1 c| + |x2 s| (for both halves of a pair at least half of it)
        pair = turn(mag, torch.ones_like(angle), self.interleaved, torch.float64).abs() + 2 * mag
        u = HALF_STEP.get(x.dtype, 2.0 ** -24)
        bound = 3 * 2.0 ** -24 * pair + u * ref.abs() * (1 + 2.0 ** -20) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
        err = (got.double() - ref).abs()
        assert (err <= bound).all(), f"{what}: off by {err.max().item():.3e}"


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("schemes", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("dim,group,rotary,interleaved", [(64, 32, 64, False), (64, 64, 32, True), (128, 32, 128, False),
                                                          (128, 64, 80, False), (128, 128, 128, True), (256, 32, 256, False),
                                                          (256, 64, 144, False), (256, 128, 16, True)])
def test_equals_append_of_turned_rows(bits, schemes, dim, group, rotary, interleaved):
    s = Setup(bits, schemes, dim, group, 2, torch.bfloat16, rotary, interleaved, seed=bits + dim + group)
    got = s.copies()
    q = s.rotary(*got, q=s.q)
    s.check_equal(got, s.reference())
    s.check_rows(q, s.q, "q")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("schemes", [(0, 0), (1, 1)])
def test_types_key_rows_and_separate_windows(dtype, interleaved, schemes):
    s = Setup(4, schemes, 128, 128, 3, DTYPES[dtype], 96, interleaved, paged=False, seed=7)
    want = s.reference()
    cache, window = s.copies()
    outs = [w.clone() for w in window]
    k_out = torch.full_like(s.k, 9.0)
    for _ in range(2):
        q = s.rotary(cache, window, q=s.q, k_out=k_out, k_window_out=outs[0], v_window_out=outs[1])
        s.check_equal((cache, outs), want)
        s.check_rows(q, s.q, "q")
        s.check_rows(k_out, s.k, "k")
    for a, b in zip(window, s.window):
        assert torch.equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (128, 128), (128, 96), (256, 256), (256, 144)])
def test_to_the_last_bit(dim, rotary, interleaved):
    """fp32 queries equal single operations bit by bit (a fused one would differ in a quarter of them), and so do the
    codes, scales and offsets of millions of 16-bit keys, of which some would differ."""
    s = Setup(4, (1, 1), dim, 32, 2, torch.float32, rotary, interleaved, old=[0], new=[1000], paged=False)
    q = s.rotary(*s.copies(), q=s.q)
    assert torch.equal(q, turn(s.q, s.table[s.position], interleaved))
    for schemes in ((1, 0), (0, 0)):
        s = Setup(4, schemes, dim, 32, 8, torch.bfloat16, rotary, interleaved, old=[0, 0], new=[4096, 1024], seed=3)
        got = s.copies()
        s.rotary(*got)
        s.check_equal(got, s.reference())


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_token_wise_without_windows(bits, dim, group):
    s = Setup(bits, (0, 0), dim, group, 2, torch.float16, dim, seed=3, windows=False)
    got = s.copies()
    assert s.rotary(*got) is None
    s.check_equal(got, s.reference())


def test_equals_the_oracles_pack():
    """One call on empty sequences against the oracle, from rows that were turned on the host."""
    s = Setup(4, (1, 0), 128, 64, 2, torch.bfloat16, 128, old=[0, 0, 0], new=[300, 128, 5])
    got = s.copies()
    s.rotary(*got)
    rows = [turn(s.k.cpu(), s.table[s.position].cpu(), False), s.v.float().cpu()]
    for which in (0, 1):
        pad = np.zeros((3, 2, s.wide * 128, 128), np.float32)
        for b, part in enumerate(rows[which].split(s.new)):
            pad[b, :, :len(part)] = part.transpose(0, 1).numpy()
        ref = orc.pack_cache(pad, s.total, 4, s.schemes[which], which, s.page_table.cpu().numpy(), s.desc.num_pages, 64)
        pages = sorted(int(s.page_table[b, j]) for b, n in enumerate(s.total) for j in range((n + 127) // 128))
        for name, a, b in zip(("codes", "scale", "zero"), got[0][which], ref):
            a = a.cpu().view(torch.uint8 if name == "codes" else torch.int16).numpy()
            assert np.array_equal(a[pages], (b if name == "codes" else b.view(np.int16))[pages]), (name, which)


def test_slices_of_a_fused_projection():
    s = Setup(4, (1, 0), 128, 128, 4, torch.bfloat16, 128, seed=5)
    want = s.reference()
    T = len(s.k)
    fused = torch.cat([s.q, s.k, s.v], 1)
    q, s.k, s.v = fused[:, :8], fused[:, 8:12], fused[:, 12:]
    got = s.copies()
    out = torch.full((T + 1, 8, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    assert s.rotary(*got, q=q, q_out=out[:T]) .data_ptr() == out.data_ptr()
    s.check_equal(got, want)
    s.check_rows(out[:T], s.q, "q")
    assert (out[T:] == 7.0).all()


def test_many_short_sequences_and_far_positions():
    """More sequences than one step of the search for a row's sequence takes, empty ones among them; positions of which
    fp32 angles would be wrong by far."""
    g = torch.Generator().manual_seed(0)
    new = torch.randint(0, 3, (1500,), generator=g).tolist()
    old = [0] * 1500
    s = Setup(4, (0, 0), 64, 64, 1, torch.bfloat16, 64, old=old, new=new, paged=False)
    got = s.copies()
    q = s.rotary(*got, q=s.q)
    s.check_equal(got, s.reference())
    s.check_rows(q, s.q, "q")
    far = 999_990
    s = Setup(4, (0, 0), 64, 64, 1, torch.bfloat16, 64, old=[far], new=[9], paged=True, windows=False)
    got = s.copies()
    q = s.rotary(*got, q=s.q)
    s.check_equal(got, s.reference())
    s.check_rows(q, s.q, "q")
    angle = (far * 10000.0 ** (-2 / 64))
    assert abs(s.table[far, 1].item() - np.cos(angle)) <= 2.0 ** -24


def test_what_is_skipped():
    """Past the table, past the pages, a negative length, a bad page, offsets that go back: reported; the sequence's
    pages, windows and turned rows are left as they were, the others' are written."""
    base = dict(old=[10, 20, 30], new=[150, 150, 150])
    kvq = Setup(4, (0, 1), 128, 128, 2, torch.bfloat16, 128, **base).kvq
    for what in ("table", "long", "negative", "page", "starts"):
        s = Setup(4, (0, 1), 128, 128, 2, torch.bfloat16, 128, **base)
        want = s.reference()
        good = [0, 2]
        if what == "table":  # sequence 2 reaches position 179
            s.table, good = s.table[:179].contiguous(), [0, 1]
        elif what == "long":
            s.lens[1] = 256 - 149
        elif what == "negative":
            s.lens[1] = -1
        elif what == "page":
            s.page_table[1] = s.desc.num_pages
        else:
            s.cu[1:3] = torch.tensor([150, 149])
        got, bad = s.copies(), ({0, 1, 2} - set(good)).pop()
        q_out, k_out = torch.full_like(s.q, 7.0), torch.full_like(s.k, 7.0)
        table = want[0] and synth.page_table_for(torch.tensor(s.total), 1, s.wide)[0]
        s.rotary(*got, q=s.q, q_out=q_out, k_out=k_out)
        assert int(s.status.item()) == (kvq.DEV_BAD_PAGE if what == "page" else kvq.DEV_BAD_SEQ_LEN)
        left = [int(p) for p in table[bad][:2]]
        for c, was, w in zip(got[0], s.cache, want[0]):
            for a, b, d in zip(c, was, w):
                assert torch.equal(a[left].view(torch.uint8), b[left].view(torch.uint8))
                if what != "starts":
                    rest = [int(p) for b_ in good for p in table[b_][:2]]
                    assert torch.equal(a[rest].view(torch.uint8), d[rest].view(torch.uint8))
        if what not in ("page", "starts"):
            rows = slice(150 * bad, 150 * bad + 150)
            assert (q_out[rows] == 7).all() and (k_out[rows] == 7).all()
            assert not (q_out == 7).all(2).all(1)[[150 * b for b in good]].any()


def test_captured_call_takes_new_lengths():
    s = Setup(2, (1, 0), 64, 32, 2, torch.float16, 64, seed=8)
    want = s.reference()
    got = s.copies()
    q_out = torch.zeros_like(s.q)
    cu = s.cu.clone()
    s.cu.zero_()
    s.rotary(*s.copies(), q=s.q, q_out=q_out)
    assert not q_out.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.rotary(*got, q=s.q, q_out=q_out)
    s.cu.copy_(cu)
    graph.replay()
    torch.cuda.synchronize()
    s.check_equal(got, want)
    s.check_rows(q_out, s.q, "q")


def test_on_another_stream_and_nothing_to_append():
    s = Setup(4, (1, 1), 128, 64, 2, torch.bfloat16, 128, seed=2)
    want, got = s.reference(), s.copies()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.rotary(*got)
    stream.synchronize()
    s.check_equal(got, want)
    s = Setup(4, (1, 0), 128, 128, 2, torch.bfloat16, 128, old=[5, 128, 300], new=[0, 0, 0])
    got = s.copies()
    assert s.rotary(*got, q=s.q).shape == (0, 4, 128)
    s.check_equal(got, (s.cache, s.window))


def test_values_that_are_refused():
    """A value that is not finite reaches its pair's other channel too; the groups of both are left zero."""
    s = Setup(4, (1, 0), 128, 64, 1, torch.bfloat16, 128, paged=False, old=[0], new=[200])
    got = s.copies()
    s.rotary(*got)
    s.check_equal(got, s.reference())
    want = s.kvq.dequant(s.desc, 0, got[0][0], 1, 200, max_blocks=s.wide)
    s.k[70, 0, 3] = float("inf")
    s.rotary(*got)
    assert int(s.status.item()) == s.kvq.DEV_NONFINITE
    k = s.kvq.dequant(s.desc, 0, got[0][0], 1, 200, max_blocks=s.wide)
    group = torch.zeros_like(k, dtype=torch.bool)
    group[:, :, 64:128, 3] = group[:, :, 64:128, 67] = True
    assert (k[group] == 0).all() and torch.equal(k[~group], want[~group])

"""Host-side checks of the append with the position rotation, of the selection of
blocks and of decode attention over lists of blocks: what is refused before
anything is launched."""
import ctypes
import math

import pytest
import torch
import torch.autograd.forward_ad as fwd

import __graft_entry__ as entry
import bit_quantized_kv_decode_gb300 as kvq
from bit_quantized_kv_decode_gb300 import _lib

P = ctypes.c_void_p
FAKE = P(0x10000)  # never read: the checks come first
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return _lib.load()


def rows(data=0x10000, st=4096, sh=128):
    return _lib.Rows(data, st, sh)


def cache(bits=4, k=1, v=0, dim=128, hkv=8, pages=64, group=0):
    return _lib.CacheDesc(bits, k, v, dim, hkv, pages, group)


def rotary(angles=0x10000, positions=4096, dim=128, interleaved=0):
    return _lib.Rotary(angles, positions, dim, interleaved)


def append(lib, c=None, dtype=0, turn=None, q=None, hq=32, k=None, v=None, batch=2, total=100, cu=FAKE, lens=FAKE, table=FAKE,
           blocks=4, windows=(FAKE,) * 4, arrays=(FAKE,) * 6, q_out=FAKE, k_out=FAKE):
    c = cache() if c is None else c
    turn = rotary() if turn is None else turn
    q, k, v = (rows() if x is None else x for x in (q, k, v))
    return lib.kvq_append_rotary(ctypes.byref(c), dtype, ctypes.byref(turn), ctypes.byref(q) if q else None, hq, ctypes.byref(k),
                                 ctypes.byref(v), batch, total, cu, lens, table, blocks, *windows, *arrays, q_out, k_out, None,
                                 None)


def select(lib, c=None, batch=2, hq=32, blocks=4, budget=4, first=1, last=1, arrays=(FAKE,) * 3, lens=FAKE, table=FAKE,
           out=(FAKE,) * 2):
    d = _lib.SelectDesc(cache() if c is None else c, batch, hq, blocks, budget, first, last)
    return lib.kvq_select_blocks(ctypes.byref(d), *arrays, lens, table, *out, None, None)


def sparse_desc(c=None, batch=2, hq=32, blocks=4, list_len=4, scale=0.0, flags=0):
    return _lib.SparseDesc(cache() if c is None else c, batch, hq, blocks, list_len, scale, flags)


def sparse(lib, q=FAKE, arrays=(FAKE,) * 6, lens=FAKE, table=FAKE, lists=(FAKE,) * 2, out=FAKE, lse=None, ws=FAKE, size=None, **kw):
    d = sparse_desc(**kw)
    if size is None:
        n = ctypes.c_size_t()
        status = lib.kvq_sparse_workspace_size(ctypes.byref(d), ctypes.byref(n))
        if status != OK:
            return status
        size = n.value
    return lib.kvq_sparse_decode_attn(ctypes.byref(d), q, *arrays, lens, table, *lists, out, lse, ws, size, None, None)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="on a GPU machine the call would launch")


@needs_no_gpu
def test_well_formed_calls_stop_at_the_device(lib):
    none = dict(q=False, q_out=None)
    assert append(lib) == DEVICE and append(lib, **none, k_out=None) == DEVICE
    assert append(lib, turn=rotary(dim=16, interleaved=1), dtype=2) == DEVICE
    assert append(lib, total=0, k=rows(None, 0, 0), v=rows(None, 0, 0), **none) == DEVICE
    assert append(lib, c=cache(k=0), windows=(None,) * 4) == DEVICE
    assert select(lib) == DEVICE and select(lib, table=None, blocks=32, hq=8, first=0, last=0) == DEVICE
    assert select(lib, blocks=16384, budget=16384, first=1, last=16383) == DEVICE
    assert sparse(lib) == DEVICE and sparse(lib, lse=FAKE, scale=0.5, hq=64, c=cache(k=0, v=1, dim=256, group=64)) == DEVICE


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(c=cache(bits=3))), (UNSUPPORTED, dict(c=cache(dim=96))), (UNSUPPORTED, dict(c=cache(group=16))),
    (INVALID, dict(dtype=3)), (INVALID, dict(batch=0)), (INVALID, dict(batch=65536)), (INVALID, dict(total=-1)),
    (INVALID, dict(blocks=0)), (INVALID, dict(table=None, blocks=33)), (INVALID, dict(cu=None)),
    (INVALID, dict(lens=P(0x10002))), (INVALID, dict(k=rows(st=4))), (INVALID, dict(v=rows(0x10008))),
    (INVALID, dict(arrays=(FAKE, FAKE, None, FAKE, FAKE, FAKE))), (INVALID, dict(windows=(None, FAKE, None, FAKE))),
    (INVALID, dict(windows=(FAKE, None, FAKE, FAKE))), (INVALID, dict(turn=rotary(None))),
    (INVALID, dict(turn=rotary(0x10004))), (INVALID, dict(turn=rotary(positions=0))), (INVALID, dict(turn=rotary(interleaved=2))),
    (UNSUPPORTED, dict(turn=rotary(dim=0))), (UNSUPPORTED, dict(turn=rotary(dim=8))), (UNSUPPORTED, dict(turn=rotary(dim=72))),
    (UNSUPPORTED, dict(turn=rotary(dim=144))), (INVALID, dict(q=False)), (INVALID, dict(q_out=None)),
    (INVALID, dict(q=rows(0x10008))), (INVALID, dict(q=rows(sh=132))), (INVALID, dict(hq=0)), (INVALID, dict(hq=65536)),
    (INVALID, dict(q_out=P(0x10008))), (INVALID, dict(k_out=P(0x10008)))])
def test_append_refusals(lib, status, kw):
    assert append(lib, **kw) == status


STEP = [(UNSUPPORTED, dict(c=cache(bits=3))), (UNSUPPORTED, dict(c=cache(dim=96))), (UNSUPPORTED, dict(c=cache(group=16))),
        (INVALID, dict(batch=0)), (INVALID, dict(batch=65536)), (INVALID, dict(hq=0)), (UNSUPPORTED, dict(hq=12)),
        (UNSUPPORTED, dict(hq=24)), (UNSUPPORTED, dict(hq=128)), (INVALID, dict(blocks=0)), (INVALID, dict(lens=None)),
        (INVALID, dict(lens=P(0x10002))), (INVALID, dict(table=P(0x10002))), (INVALID, dict(table=None, blocks=33))]


@pytest.mark.parametrize("status,kw", STEP + [
    (UNSUPPORTED, dict(c=cache(k=0))), (UNSUPPORTED, dict(blocks=16385)), (INVALID, dict(budget=0)), (INVALID, dict(first=-1)),
    (INVALID, dict(last=-1)), (INVALID, dict(first=3, last=2)), (INVALID, dict(first=2 ** 31 - 1, last=2 ** 31 - 1)),
    (UNSUPPORTED, dict(budget=2 ** 27)), (INVALID, dict(arrays=(None, FAKE, FAKE))), (INVALID, dict(arrays=(P(0x10008), FAKE, FAKE))),
    (INVALID, dict(arrays=(FAKE, FAKE, None))), (INVALID, dict(out=(None, FAKE))), (INVALID, dict(out=(FAKE, None))),
    (INVALID, dict(out=(P(0x10002), FAKE)))])
def test_select_refusals(lib, status, kw):
    assert select(lib, **kw) == status


@pytest.mark.parametrize("status,kw", STEP + [
    (UNSUPPORTED, dict(blocks=(1 << 23) + 1)), (INVALID, dict(list_len=0)), (UNSUPPORTED, dict(list_len=2 ** 27)),
    (INVALID, dict(scale=math.nan)), (INVALID, dict(scale=math.inf)), (INVALID, dict(flags=2)), (INVALID, dict(flags=8)), (INVALID, dict(q=None)),
    (INVALID, dict(q=P(0x10008))), (INVALID, dict(arrays=(None,) + (FAKE,) * 5)),
    (INVALID, dict(arrays=(FAKE,) * 5 + (P(0x10008),))), (INVALID, dict(lists=(None, FAKE))), (INVALID, dict(lists=(FAKE, None))),
    (INVALID, dict(lists=(P(0x10001), FAKE))), (INVALID, dict(out=None)), (INVALID, dict(out=P(0x10008))),
    (INVALID, dict(lse=P(0x10002))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=P(0x10010))), (WORKSPACE, dict(size=255))])
def test_sparse_refusals(lib, status, kw):
    assert sparse(lib, **kw) == status


def test_null_descriptors(lib):
    r, n, c = rows(), ctypes.c_size_t(), cache()
    assert lib.kvq_append_rotary(ctypes.byref(c), 0, None, None, 0, r, r, 2, 100, FAKE, FAKE, FAKE, 4, *([FAKE] * 10), None, None,
                                 None, None) == INVALID
    assert lib.kvq_append_rotary(None, 0, rotary(), None, 0, r, r, 2, 100, FAKE, FAKE, FAKE, 4, *([FAKE] * 10), None, None,
                                 None, None) == INVALID
    assert lib.kvq_select_blocks(None, *([FAKE] * 7), None, None) == INVALID
    assert lib.kvq_sparse_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.kvq_sparse_workspace_size(ctypes.byref(sparse_desc()), None) == INVALID
    assert lib.kvq_sparse_decode_attn(None, *([FAKE] * 13), None, 0, None, None) == INVALID


@pytest.mark.parametrize("batch,per,list_len", [(1, 1, 1), (1, 4, 2), (4, 4, 500), (1, 8, 8192), (1, 1, 100000), (65535, 4, 64)])
def test_workspace_is_of_the_ranges_and_bounded(lib, batch, per, list_len):
    """One fp32 row of 128 channels and one lse per range and query head, in two parts of whole 256 bytes: never more
    ranges than entries, and not many times more than the device runs at a time."""
    size = kvq.sparse_workspace_size(cache(), batch, 8 * per, list_len)
    lists = batch * 8
    most = min(list_len, 32 * 152 // lists + 2) * lists * per
    assert size <= most * 129 * 4 + 512
    if list_len == 1 or lists > 33 * 152:  # one range a list: nothing to keep
        assert size == 0
    if list_len >= 500 and batch < 65535:
        assert size >= 2 * lists * per * 129 * 4


def test_rotary_table():
    t = kvq.rotary_table(70000, 32, 500000.0, device="cpu")
    p = torch.tensor([0, 1, 69999], dtype=torch.float64)
    a = p[:, None] * 500000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    assert t.shape == (70000, 32) and t.dtype == torch.float32
    assert torch.equal(t[[0, 1, 69999]], torch.cat([a.cos(), a.sin()], 1).float())
    for dim in (0, 15, -2):
        with pytest.raises(ValueError, match="even"):
            kvq.rotary_table(8, dim, device="cpu")


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    desc = kvq.cache_desc(4, 1, 0, 8, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.append_rotary(desc, torch.zeros(8, 128), x, x, cu, cu[:1], None, None, max_blocks=1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.select_blocks(desc, x, None, cu[:1], 1, max_blocks=1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.sparse_decode_attn(desc, x, None, None, cu[:1], cu, cu, max_blocks=1)


class Given:
    """One well-formed call of each."""

    def __init__(self):
        B, self.T, self.H, D = 2, 6, 2, 128
        g = torch.Generator(device="cuda").manual_seed(1)
        self.desc = kvq.cache_desc(4, 1, 0, self.H, 4)
        self.caches = [kvq.alloc_cache(self.desc) for _ in "kv"]
        for c in self.caches:
            for t in c:
                t.zero_()
        self.rows = torch.randn(self.T, 8, D, generator=g, device="cuda").to(torch.bfloat16)
        self.k, self.v = self.rows[:, 4:6], self.rows[:, 6:]
        self.q = self.rows[:B].contiguous()
        self.table = kvq.rotary_table(300, 128)
        self.cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor([130, 255], dtype=torch.int32, device="cuda")
        self.window = [torch.zeros(B, self.H, 128, D, device="cuda") for _ in "kv"]
        self.blocks = torch.zeros(B, self.H, 32, dtype=torch.int32, device="cuda")
        self.counts = torch.ones(B, self.H, dtype=torch.int32, device="cuda")

    def append(self, **kw):
        a = dict(table=self.table, k_new=self.k, v_new=self.v, cu_seqlens=self.cu, seq_lens=self.lens - 4, k_cache=self.caches[0],
                 v_cache=self.caches[1], k_window=self.window[0], v_window=self.window[1], max_blocks=2)
        return kvq.append_rotary(self.desc, **{**a, **kw})

    def select(self, desc=None, **kw):
        a = dict(q=self.q, k_cache=self.caches[0], seq_lens=self.lens, budget=2, max_blocks=2)
        return kvq.select_blocks(desc or self.desc, **{**a, **kw})

    def sparse(self, **kw):
        a = dict(q=self.q, k_cache=self.caches[0], v_cache=self.caches[1], seq_lens=self.lens, blocks=self.blocks,
                 counts=self.counts, max_blocks=2)
        return kvq.sparse_decode_attn(self.desc, **{**a, **kw})


@pytest.mark.gpu
def test_wrappers_refuse_bad_tensors():
    g = Given()
    half, wide = g.q.half(), torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    short = (g.caches[0][0], g.caches[0][1][:3], g.caches[0][2])
    bad = [lambda: g.append(table=g.table.half()), lambda: g.append(table=g.table[:, :64]), lambda: g.append(table=g.table.cpu()),
           lambda: g.append(table=g.table[0]), lambda: g.append(table=g.table.clone().requires_grad_()),
           lambda: g.append(q=g.rows.half()), lambda: g.append(q=g.rows[:5]), lambda: g.append(q=g.rows[..., :64]),
           lambda: g.append(q=g.rows.clone().requires_grad_()), lambda: g.append(q_out=torch.empty_like(g.rows)),
           lambda: g.append(q=g.rows, q_out=torch.empty_like(g.rows[:, :4])),
           lambda: g.append(q=g.rows, q_out=torch.empty_like(g.rows).half()), lambda: g.append(k_out=torch.empty_like(g.rows)),
           lambda: g.append(k_out=torch.empty(g.T, 128, g.H, dtype=torch.bfloat16, device="cuda").transpose(1, 2)),
           lambda: g.append(k_window=None), lambda: g.append(k_new=g.k.float()), lambda: g.append(k_new=g.k.clone().requires_grad_()),
           lambda: g.append(max_blocks=None), lambda: g.append(k_cache=short), lambda: g.append(seq_lens=None),
           lambda: g.select(q=half), lambda: g.select(q=g.q[0]), lambda: g.select(q=wide[::2]), lambda: g.select(q=g.q[..., :64]),
           lambda: g.select(q=g.q.clone().requires_grad_()), lambda: g.select(budget=0), lambda: g.select(first=1 << 32), lambda: g.select(last=1 << 32),
           lambda: g.select(seq_lens=g.lens[:1]),
           lambda: g.select(seq_lens=None), lambda: g.select(max_blocks=None), lambda: g.select(k_cache=short),
           lambda: g.select(blocks=g.blocks.long()), lambda: g.select(counts=g.counts[:1]),
           lambda: g.select(page_table=g.blocks[:, 0].long()),
           lambda: g.sparse(q=half), lambda: g.sparse(q=wide[::2]), lambda: g.sparse(q=g.q.clone().requires_grad_()),
           lambda: g.sparse(blocks=g.blocks[:1]), lambda: g.sparse(blocks=g.blocks.long()), lambda: g.sparse(blocks=g.blocks[:, :, ::2]),
           lambda: g.sparse(counts=None), lambda: g.sparse(counts=g.counts.cpu()), lambda: g.sparse(v_cache=short),
           lambda: g.sparse(out=torch.empty_like(half)), lambda: g.sparse(lse=torch.zeros(2, 7, device="cuda")),
           lambda: g.sparse(workspace=torch.zeros(1 << 20, device="cuda")), lambda: g.sparse(max_blocks=None)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: g.append(table=kvq.rotary_table(300, 24)), lambda: g.append(table=kvq.rotary_table(300, 144)),
                 lambda: g.select(first=2), lambda: g.select(desc=kvq.cache_desc(4, 0, 0, 2, 4)),
                 lambda: g.select(q=wide[:2, :6].contiguous()), lambda: g.sparse(sm_scale=math.inf)):
        with pytest.raises(kvq.KvqError):
            call()
    with torch.no_grad():
        g.append(table=g.table.clone().requires_grad_(), q=g.rows.clone().requires_grad_())
        g.select(q=g.q.clone().requires_grad_())
    with fwd.dual_level():
        def dual(x):
            return fwd.make_dual(x, torch.ones_like(x))

        for call in (lambda: g.append(table=dual(g.table)), lambda: g.append(q=dual(g.rows)), lambda: g.append(k_new=dual(g.k)),
                     lambda: g.select(q=dual(g.q)), lambda: g.sparse(q=dual(g.q))):
            with pytest.raises(ValueError, match="tangent"):
                call()


@pytest.mark.gpu
def test_wrappers_refuse_outputs_over_other_arrays():
    g = Given()
    own, kept = g.rows.contiguous(), torch.zeros(4 * g.T * 8 * 128, dtype=torch.bfloat16, device="cuda")
    n, m = g.T * 8 * 128, g.T * 2 * 128
    q_out, over, apart = kept[:n].view(g.T, 8, 128), kept[n - 8:n - 8 + m].view(g.T, 2, 128), kept[n:n + m].view(g.T, 2, 128)
    window = g.window[0].view(torch.bfloat16).view(-1)[:m].view(g.T, 2, 128)
    codes = g.caches[0][0].view(-1)[:m * 2].view(torch.bfloat16).view(g.T, 2, 128)
    ints = torch.zeros(64, dtype=torch.int32, device="cuda")
    lists, numbers = ints[:8].view(2, 2, 2), ints[4:8].view(2, 2)
    size = kvq.sparse_workspace_size(g.desc, 2, 8, 32)
    assert size > 0
    memory = torch.zeros(size + 8192, dtype=torch.uint8, device="cuda")

    def out(at):
        return memory[at:at + 4096].view(torch.bfloat16).view(2, 8, 128)

    def lse(at):
        return memory[at:at + 64].view(torch.float32).view(2, 8)

    bad = [lambda: g.append(q=own, q_out=own), lambda: g.append(q=g.rows, q_out=q_out, k_out=over), lambda: g.append(k_out=window),
           lambda: g.append(k_out=codes), lambda: g.append(k_new=apart, k_out=apart),
           lambda: g.append(v_new=over, k_out=apart), lambda: g.append(k_new=own[:, :2], q=g.rows, q_out=own),
           lambda: g.select(blocks=lists, counts=numbers), lambda: g.select(blocks=lists, seq_lens=ints[6:8]),
           lambda: g.select(counts=numbers, seq_lens=ints[7:9]),
           lambda: g.select(q=memory[:4096].view(torch.bfloat16).view(2, 8, 128), blocks=memory[4064:4096].view(torch.int32).view(2, 2, 2)),
           lambda: g.sparse(q=out(0), out=out(4080)), lambda: g.sparse(out=out(0), lse=lse(4080)),
           lambda: g.sparse(out=out(size - 16), workspace=memory[:size]), lambda: g.sparse(lse=lse(size - 16), workspace=memory[:size]),
           lambda: g.sparse(q=out(size - 16), workspace=memory[:size]),
           lambda: g.sparse(out=g.caches[1][0].view(-1)[:4096].view(torch.bfloat16).view(2, 8, 128)),
           lambda: g.sparse(blocks=memory[:32].view(torch.int32).view(2, 2, 2), lse=lse(16))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps"):
            call()
            pytest.fail(f"call {i} was not refused")
    assert (memory == 0).all() and (kept == 0).all() and (ints == 0).all()
    turned = g.append(q=g.rows, q_out=q_out, k_out=apart)  # right behind one another
    assert turned is q_out and torch.equal(turned[:, 4:6], apart)
    g.select(blocks=lists, counts=ints[8:12].view(2, 2))
    want = g.sparse()
    assert torch.equal(g.sparse(out=out(size), lse=lse(size + 4096), workspace=memory)[0], want)

"""Host-side checks of the operators over rows of new tokens (no GPU needed):
descriptors, pointers, strides and sizes that are refused before anything is
launched, and the wrappers' checks of their tensors."""
import ctypes

import pytest
import torch

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


def prompt(lib, q=None, k=None, v=None, cu=FAKE, out=FAKE, lse=None, dtype=0, dim=128, hq=32, hkv=8, batch=2, total=100,
           causal=1, scale=0.0, flags=0):
    d = _lib.PromptDesc(dtype, dim, hq, hkv, batch, total, causal, scale, flags)
    q, k, v = (rows() if x is None else x for x in (q, k, v))
    return lib.kvq_prompt_attn(ctypes.byref(d), ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), cu, out, lse, None,
                               None)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="on a GPU machine the call would launch")


@needs_no_gpu
def test_well_formed_calls_stop_at_the_device(lib):
    assert prompt(lib) == DEVICE
    assert prompt(lib, dim=256, dtype=1, hq=24, causal=0, lse=FAKE) == DEVICE
    assert prompt(lib, total=0, q=rows(None, 0, 0), k=rows(None, 0, 0), v=rows(None, 0, 0), out=None) == DEVICE
    assert append(lib) == DEVICE
    assert chunk(lib) == DEVICE


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(dim=96)), (UNSUPPORTED, dict(dim=512)), (UNSUPPORTED, dict(hq=20)), (UNSUPPORTED, dict(hq=136)),
    (UNSUPPORTED, dict(dtype=2)), (INVALID, dict(dtype=3)), (INVALID, dict(dtype=-1)), (INVALID, dict(hkv=0)),
    (INVALID, dict(batch=0)), (INVALID, dict(batch=65536)), (INVALID, dict(total=-1)),
    (UNSUPPORTED, dict(total=2 ** 31 - 1)), (INVALID, dict(causal=2)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(flags=4)), (INVALID, dict(cu=None)), (INVALID, dict(out=None)),
    (INVALID, dict(out=P(0x10008))), (INVALID, dict(cu=P(0x10002))), (INVALID, dict(lse=P(0x10002))),
    (INVALID, dict(q=rows(None))), (INVALID, dict(k=rows(0x10008))), (INVALID, dict(v=rows(st=4))),
    (INVALID, dict(v=rows(sh=0))), (INVALID, dict(q=rows(st=-4096))), (INVALID, dict(k=rows(sh=132))),
    (INVALID, dict(k=rows(st=1 << 37)))])
def test_prompt_refusals(lib, status, kw):
    assert prompt(lib, **kw) == status


def cache(bits=4, k=1, v=0, dim=128, hkv=8, pages=64, group=0):
    return _lib.CacheDesc(bits, k, v, dim, hkv, pages, group)


def append(lib, c=None, dtype=0, k=None, v=None, batch=2, total=100, cu=FAKE, lens=FAKE, table=FAKE, blocks=4,
           windows=(FAKE,) * 4, arrays=(FAKE,) * 6):
    c = cache() if c is None else c
    k, v = (rows() if x is None else x for x in (k, v))
    return lib.kvq_append_chunk(ctypes.byref(c), dtype, ctypes.byref(k), ctypes.byref(v), batch, total, cu, lens, table,
                                blocks, *windows, *arrays, None, None)


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(c=cache(bits=3))), (UNSUPPORTED, dict(c=cache(dim=96))), (INVALID, dict(c=cache(k=2))),
    (INVALID, dict(dtype=3)), (INVALID, dict(batch=0)), (INVALID, dict(batch=65536)), (INVALID, dict(total=-1)),
    (INVALID, dict(blocks=0)), (INVALID, dict(table=None, blocks=33)), (INVALID, dict(cu=None)), (INVALID, dict(lens=None)),
    (INVALID, dict(lens=P(0x10002))), (INVALID, dict(table=P(0x10001))), (INVALID, dict(k=rows(st=4))),
    (INVALID, dict(dtype=2, v=rows(st=4098))), (INVALID, dict(arrays=(FAKE, FAKE, None, FAKE, FAKE, FAKE))),
    (INVALID, dict(arrays=(FAKE, FAKE, FAKE, P(0x10008), FAKE, FAKE))),
    (INVALID, dict(windows=(None, FAKE, None, FAKE))),   # K is channel-wise: its window is needed
    (INVALID, dict(windows=(FAKE, FAKE, None, FAKE))),   # a window without its output
    (INVALID, dict(windows=(FAKE, None, FAKE, FAKE))),   # an output without its window
    (INVALID, dict(windows=(P(0x10004), FAKE, FAKE, FAKE)))])
def test_append_chunk_refusals(lib, status, kw):
    assert append(lib, **kw) == status


def chunk_desc(c=None, dtype=0, batch=2, total=100, hq=32, blocks=4, causal=1, scale=0.0, flags=0):
    return _lib.ChunkDesc(cache() if c is None else c, dtype, batch, total, hq, blocks, causal, scale, flags)


def chunk(lib, q=None, arrays=(FAKE,) * 6, cu=FAKE, lens=FAKE, table=FAKE, out=FAKE, lse=None, ws=FAKE, size=None, **kw):
    d = chunk_desc(**kw)
    n = ctypes.c_size_t()
    if size is None:
        st = lib.kvq_chunk_workspace_size(ctypes.byref(d), ctypes.byref(n))
        if st != OK:
            return st
        size = n.value
    q = rows() if q is None else q
    return lib.kvq_chunk_attn(ctypes.byref(d), ctypes.byref(q), *arrays, cu, lens, table, out, lse, ws, size, None, None)


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(c=cache(group=16))), (UNSUPPORTED, dict(hq=20)), (UNSUPPORTED, dict(hq=136)),
    (UNSUPPORTED, dict(dtype=2)), (INVALID, dict(dtype=5)), (INVALID, dict(batch=0)), (INVALID, dict(total=-1)),
    (UNSUPPORTED, dict(total=2 ** 31 - 1)), (INVALID, dict(blocks=0)), (UNSUPPORTED, dict(blocks=(1 << 23) + 1)),
    (INVALID, dict(causal=-1)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(flags=2)),
    (INVALID, dict(table=None, blocks=33)), (INVALID, dict(q=rows(sh=4))), (INVALID, dict(q=rows(0x10002))),
    (INVALID, dict(arrays=(None,) + (FAKE,) * 5)), (INVALID, dict(arrays=(FAKE,) * 5 + (P(0x10008),))),
    (INVALID, dict(cu=None)), (INVALID, dict(lens=None)), (INVALID, dict(out=None)), (INVALID, dict(lse=P(0x10002))),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=P(0x10010))), (WORKSPACE, dict(size=255))])
def test_chunk_refusals(lib, status, kw):
    assert chunk(lib, **kw) == status


def test_null_descriptors(lib):
    r, n = rows(), ctypes.c_size_t()
    assert lib.kvq_prompt_attn(None, r, r, r, FAKE, FAKE, None, None, None) == INVALID
    assert lib.kvq_chunk_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.kvq_chunk_workspace_size(ctypes.byref(chunk_desc()), None) == INVALID
    assert lib.kvq_append_chunk(None, 0, r, r, 1, 1, FAKE, FAKE, FAKE, 1, *([FAKE] * 10), None, None) == INVALID


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.prompt_attn(x, x, x, cu)
    desc = kvq.cache_desc(4, 0, 0, 8, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.append_chunk(desc, x, x, cu, cu[:1], None, None, max_blocks=1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.chunk_attn(desc, x, None, None, cu, cu[:1], max_blocks=1)


@pytest.mark.gpu
def test_wrappers_refuse_bad_tensors():
    T, D = 6, 128
    q = torch.zeros(T, 8, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(T, 2, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 1, 0, 2, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    window = torch.zeros(1, 2, 128, D, device="cuda")
    bad = [lambda: kvq.prompt_attn(q.float(), k, k, cu), lambda: kvq.prompt_attn(q, k.half(), k, cu),
           lambda: kvq.prompt_attn(q, k[:5], k, cu), lambda: kvq.prompt_attn(q, k, k[:, :1], cu),
           lambda: kvq.prompt_attn(q, k, k, cu.long()), lambda: kvq.prompt_attn(q, k, k, cu[:1]),
           lambda: kvq.prompt_attn(q, k, k, cu, out=torch.empty_like(k)),
           lambda: kvq.prompt_attn(q, k, k, cu, out=torch.empty_like(q.half())),
           lambda: kvq.prompt_attn(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu),
           lambda: kvq.prompt_attn(q, k[:1].expand(T, 2, D), k, cu),
           lambda: kvq.prompt_attn(q, k[:, :1].expand(T, 2, D), k, cu),
           lambda: kvq.prompt_attn(q.clone().requires_grad_(), k, k, cu),
           lambda: kvq.prompt_attn(q, k, k, cu.cpu()),
           lambda: kvq.append_chunk(desc, k, k, cu, lens, *caches, max_blocks=1),
           lambda: kvq.append_chunk(desc, k, k, cu, lens, *caches, window, window),
           lambda: kvq.append_chunk(desc, k, k.float(), cu, lens, *caches, window, window, max_blocks=1),
           lambda: kvq.append_chunk(desc, q, q, cu, lens, *caches, window, window, max_blocks=1),
           lambda: kvq.append_chunk(desc, k, k, cu, lens, *caches, window[:, :1], window, max_blocks=1),
           lambda: kvq.append_chunk(desc, k, k, cu, lens[:0], *caches, window, window, max_blocks=1),
           lambda: kvq.chunk_attn(desc, q, *caches, cu, lens),
           lambda: kvq.chunk_attn(desc, q[..., :64], *caches, cu, lens, max_blocks=1),
           lambda: kvq.chunk_attn(desc, q.clone().requires_grad_(), *caches, cu, lens, max_blocks=1),
           lambda: kvq.chunk_attn(desc, q, caches[0][:2] + (caches[0][2][..., :4],), caches[1], cu, lens, max_blocks=1)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(kvq.KvqError):  # 4 query heads per KV head times 17
        kvq.prompt_attn(torch.zeros(T, 34, D, dtype=torch.bfloat16, device="cuda"), k, k, cu)
    with torch.no_grad():
        kvq.prompt_attn(q.clone().requires_grad_(), k, k, cu)
    empty = kvq.prompt_attn(q[:0], k[:0], k[:0], torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert empty.shape == (0, 8, D)


@pytest.mark.gpu
def test_wrappers_refuse_outputs_over_their_inputs():
    T, D = 6, 128
    qkv = torch.zeros(T, 12, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 1, 1, 2, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    window, other = (torch.zeros(1, 2, 128, D, device="cuda") for _ in "kv")
    inside = qkv.view(-1)[-T * 8 * D:].view(T, 8, D)
    own = q.contiguous()
    bad = [lambda: kvq.prompt_attn(q, k, v, cu, out=inside), lambda: kvq.prompt_attn(own, k, v, cu, out=own),
           lambda: kvq.prompt_attn(q, k, v, cu, lse=qkv.view(torch.float32).view(-1)[:T * 8].view(T, 8)),
           lambda: kvq.chunk_attn(desc, own, *caches, cu, lens, max_blocks=1, out=own),
           lambda: kvq.append_chunk(desc, k, v, cu, lens, *caches, window, window, max_blocks=1),
           lambda: kvq.append_chunk(desc, k, v, cu, lens, *caches, window, other, max_blocks=1, k_window_out=other)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps|same memory"):
            call()
            pytest.fail(f"call {i} was not refused")
    out = torch.full((T + 1, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kvq.prompt_attn(own, k, v, cu, out=out[:T]).abs().max().item() == 0.0
    assert (out[T:] == 7.0).all()

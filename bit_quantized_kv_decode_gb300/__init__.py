"""Decode attention over an INT2/INT4 group-quantized KV cache on GB300.

Thin PyTorch-facing wrappers over the C-ABI of ``libkvq.so`` (include/kvq.h):
they check tensor dtypes, devices and shapes, pass raw device pointers and the
current CUDA stream, and raise on a non-OK status.  Every step of the
computation runs in the library's CUDA kernels; there is no other code path.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import (CHANNELWISE, DEV_BAD_PAGE, DEV_BAD_SEQ_LEN, DEV_NONFINITE, DEV_TIMEOUT, FLAG_E2M1_V, FLAG_TEST_STALL,
                   FLAG_TEST_STALL_MMA, OPERANDS_BF16, OPERANDS_FP8, TOKENWISE, AttnDesc, CacheDesc, ChunkDesc, KvqError, PromptDesc, Rows)

BLOCK_TOKENS = 128
HEAD_DIM = 128
GROUP_Q = 4

__all__ = ["CacheDesc", "AttnDesc", "KvqError", "TOKENWISE", "CHANNELWISE", "OPERANDS_FP8", "OPERANDS_BF16",
           "DEV_BAD_SEQ_LEN", "DEV_BAD_PAGE", "DEV_NONFINITE", "DEV_TIMEOUT", "FLAG_TEST_STALL", "FLAG_TEST_STALL_MMA",
           "FLAG_E2M1_V", "cache_desc", "attn_desc", "cache_bytes", "block_bytes", "sz_per_block", "alloc_cache", "pack",
           "append", "dequant", "workspace_size", "decode_attn", "decode_attn_static", "merge", "library",
           "prompt_attn", "append_chunk", "chunk_workspace_size", "chunk_attn"]


def library() -> ctypes.CDLL:
    return _lib.load()


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=None, numel=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def cache_desc(bits: int, k_scheme: int, v_scheme: int, num_kv_heads: int, num_pages: int,
               head_dim: int = HEAD_DIM, group: int = 128) -> CacheDesc:
    return CacheDesc(bits, k_scheme, v_scheme, head_dim, num_kv_heads, num_pages, group)


def attn_desc(cache: CacheDesc, batch: int, max_blocks: int, mode: int = OPERANDS_FP8, sm_scale: float = 0.0,
              num_ctas: int = 0, flags: int = 0, num_q_heads: Optional[int] = None) -> AttnDesc:
    hq = GROUP_Q * cache.num_kv_heads if num_q_heads is None else num_q_heads
    return AttnDesc(cache, batch, hq, max_blocks, mode, sm_scale, num_ctas, flags)


def block_bytes(bits: int, head_dim: int = HEAD_DIM) -> int:
    return BLOCK_TOKENS * head_dim * bits // 8


def sz_per_block(desc: CacheDesc) -> int:
    """s (or z) values per page and KV head: 128 * head_dim / group."""
    return BLOCK_TOKENS * desc.head_dim // (desc.group_size or 128)


def cache_bytes(desc: CacheDesc) -> Tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check(library().kvq_cache_bytes(ctypes.byref(desc), ctypes.byref(cb), ctypes.byref(sb)), "kvq_cache_bytes")
    return cb.value, sb.value


def alloc_cache(desc: CacheDesc, device="cuda"):
    """Zeroed (codes, scale, zero) arrays for one K or V cache."""
    P, H = desc.num_pages, desc.num_kv_heads
    codes = torch.zeros(P, H, block_bytes(desc.bits, desc.head_dim), dtype=torch.uint8, device=device)
    scale = torch.zeros(P, H, sz_per_block(desc), dtype=torch.float16, device=device)
    zero = torch.zeros(P, H, sz_per_block(desc), dtype=torch.float16, device=device)
    return codes, scale, zero


def _geometry(batch, max_seq_len, seq_lens, page_table, max_blocks):
    need = (max_seq_len + BLOCK_TOKENS - 1) // BLOCK_TOKENS
    if page_table is not None:
        _need(page_table, "page_table", torch.int32)
        if page_table.dim() != 2 or page_table.shape[0] != batch:
            raise ValueError("page_table must be int32 [batch, max_blocks]")
        mb = page_table.shape[1]
    else:
        mb = max_blocks if max_blocks is not None else need
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, batch)
    return mb


def pack(desc: CacheDesc, which: int, x: torch.Tensor, seq_lens: Optional[torch.Tensor] = None,
         page_table: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None, cache=None,
         dev_status: Optional[torch.Tensor] = None):
    """Quantize + pack fp32 x [B, Hkv, L, head_dim] into a K (which=0) or V
    (which=1) cache; returns (codes, scale, zero)."""
    _need(x, "x", torch.float32)
    if x.dim() != 4 or x.shape[1] != desc.num_kv_heads or x.shape[3] != desc.head_dim:
        raise ValueError("x must be fp32 [batch, num_kv_heads, max_seq_len, head_dim]")
    B, _, L, _ = x.shape
    mb = _geometry(B, L, seq_lens, page_table, max_blocks)
    codes, scale, zero = cache if cache is not None else alloc_cache(desc, x.device)
    _need(codes, "codes", torch.uint8)
    _need(scale, "scale", (torch.float16, torch.int16, torch.uint16))
    _need(zero, "zero", (torch.float16, torch.int16, torch.uint16))
    if dev_status is not None:
        _need(dev_status, "dev_status", (torch.int32, torch.uint32), 1)
    st = library().kvq_pack(ctypes.byref(desc), which, _p(x), B, L, _p(seq_lens), _p(page_table), mb, _p(codes),
                            _p(scale), _p(zero), _p(dev_status), _stream())
    _lib.check(st, "kvq_pack")
    return codes, scale, zero


def append(desc: CacheDesc, which: int, x_new: torch.Tensor, seq_lens: torch.Tensor, cache, window: torch.Tensor,
           page_table: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None,
           dev_status: Optional[torch.Tensor] = None):
    """Append fp32 x_new [B, Hkv, 128] at positions seq_lens (tokens already
    cached) to a packed K (which=0) or V (which=1) cache, through the caller's
    fp32 window [B, Hkv, 128, 128] of each current block; returns the cache.
    The caller advances seq_lens afterwards."""
    _need(x_new, "x_new", torch.float32)
    _need(window, "window", torch.float32)
    _need(seq_lens, "seq_lens", torch.int32)
    if x_new.dim() != 3 or x_new.shape[1] != desc.num_kv_heads or x_new.shape[2] != desc.head_dim:
        raise ValueError("x_new must be fp32 [batch, num_kv_heads, head_dim]")
    B = x_new.shape[0]
    if tuple(window.shape) != (B, desc.num_kv_heads, BLOCK_TOKENS, desc.head_dim):
        raise ValueError("window must be fp32 [batch, num_kv_heads, 128, head_dim]")
    if seq_lens.numel() != B:
        raise ValueError("seq_lens must hold one int32 per sequence")
    if page_table is not None:
        _need(page_table, "page_table", torch.int32)
        mb = page_table.shape[1]
    elif max_blocks is not None:
        mb = int(max_blocks)
    else:
        raise ValueError("append needs page_table or max_blocks")
    codes, scale, zero = cache
    if dev_status is not None:
        _need(dev_status, "dev_status", (torch.int32, torch.uint32), 1)
    st = library().kvq_append(ctypes.byref(desc), which, _p(x_new), B, _p(seq_lens), _p(page_table), mb,
                              _p(window), _p(codes), _p(scale), _p(zero), _p(dev_status), _stream())
    _lib.check(st, "kvq_append")
    return cache


def dequant(desc: CacheDesc, which: int, cache, batch: int, max_seq_len: int,
            seq_lens: Optional[torch.Tensor] = None, page_table: Optional[torch.Tensor] = None,
            max_blocks: Optional[int] = None, dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x_hat fp32 [B, Hkv, L, 128] read back from a packed cache."""
    codes, scale, zero = cache
    mb = _geometry(batch, max_seq_len, seq_lens, page_table, max_blocks)
    out = torch.empty(batch, desc.num_kv_heads, max_seq_len, desc.head_dim, dtype=torch.float32, device=codes.device)
    st = library().kvq_dequant(ctypes.byref(desc), which, _p(codes), _p(scale), _p(zero), batch, max_seq_len,
                               _p(seq_lens), _p(page_table), mb, _p(out), _p(dev_status), _stream())
    _lib.check(st, "kvq_dequant")
    return out


def workspace_size(desc: AttnDesc) -> int:
    n = ctypes.c_size_t()
    _lib.check(library().kvq_decode_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "kvq_decode_workspace_size")
    return n.value


def decode_path(desc: AttnDesc) -> int:
    """The decode kernel a call with this descriptor runs: _lib.PATH_SPECIALISED
    or _lib.PATH_GENERAL (kvq_decode_path)."""
    n = ctypes.c_int32()
    _lib.check(library().kvq_decode_path(ctypes.byref(desc), ctypes.byref(n)), "kvq_decode_path")
    return n.value


def decode_attn(desc: CacheDesc, q: torch.Tensor, k_cache, v_cache, seq_lens: torch.Tensor,
                page_table: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None,
                mode: int = OPERANDS_FP8, sm_scale: float = 0.0, num_ctas: int = 0,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                flags: int = 0):
    """out fp32 [B, Hq, 128] and lse fp32 [B, Hq] for bf16 q [B, Hq, 128]."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[2] != desc.head_dim:
        raise ValueError("q must be bf16 [batch, num_q_heads, head_dim]")
    B, Hq, _ = q.shape
    if page_table is not None:
        mb = _geometry(B, 1, seq_lens, page_table, None)
    else:
        if max_blocks is None:
            raise ValueError("max_blocks is required for a contiguous cache")
        mb = max_blocks
        _need(seq_lens, "seq_lens", torch.int32, B)
    ad = AttnDesc(desc, B, Hq, mb, mode, sm_scale, num_ctas, flags)
    if out is None:
        out = torch.empty(B, Hq, desc.head_dim, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, B * Hq * desc.head_dim)
    _need(lse, "lse", torch.float32, B * Hq)
    if workspace is None:
        workspace = torch.empty(workspace_size(ad), dtype=torch.uint8, device=q.device)
    kc, ks, kz = k_cache
    vc, vs, vz = v_cache
    st = library().kvq_decode_attn(ctypes.byref(ad), _p(q), _p(kc), _p(ks), _p(kz), _p(vc), _p(vs), _p(vz),
                                   _p(seq_lens), _p(page_table), _p(out), _p(lse), _p(workspace),
                                   workspace.numel(), _p(dev_status), _stream())
    _lib.check(st, "kvq_decode_attn")
    return out, lse


def decode_attn_static(desc: CacheDesc, q: torch.Tensor, k_cache, v_cache, seq_lens: torch.Tensor,
                       page_table: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None,
                       mode: int = OPERANDS_FP8, sm_scale: float = 0.0, num_ctas: int = 0,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       dev_status: Optional[torch.Tensor] = None):
    """decode_attn for callers that cannot allocate device memory: the C entry
    point keeps its scratch in a fixed device array owned by the library (see
    kvq_decode_attn_static in include/kvq.h).  `out` and `lse` are still
    caller buffers; pass them preallocated to avoid any allocation here."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[2] != desc.head_dim:
        raise ValueError("q must be bf16 [batch, num_q_heads, head_dim]")
    B, Hq, _ = q.shape
    if page_table is not None:
        mb = _geometry(B, 1, seq_lens, page_table, None)
    else:
        if max_blocks is None:
            raise ValueError("max_blocks is required for a contiguous cache")
        mb = max_blocks
        _need(seq_lens, "seq_lens", torch.int32, B)
    ad = AttnDesc(desc, B, Hq, mb, mode, sm_scale, num_ctas, 0)
    if out is None:
        out = torch.empty(B, Hq, desc.head_dim, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, B * Hq * desc.head_dim)
    _need(lse, "lse", torch.float32, B * Hq)
    kc, ks, kz = k_cache
    vc, vs, vz = v_cache
    st = library().kvq_decode_attn_static(ctypes.byref(ad), _p(q), _p(kc), _p(ks), _p(kz), _p(vc), _p(vs), _p(vz),
                                          _p(seq_lens), _p(page_table), _p(out), _p(lse), _p(dev_status),
                                          _stream())
    _lib.check(st, "kvq_decode_attn_static")
    return out, lse


def merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, out: Optional[torch.Tensor] = None,
          lse: Optional[torch.Tensor] = None):
    """Log-sum-exp merge of fp32 o_parts [R, S, D] / lse_parts [R, S]."""
    _need(o_parts, "o_parts", torch.float32)
    _need(lse_parts, "lse_parts", torch.float32)
    R, S, D = o_parts.shape
    if out is None:
        out = torch.empty(R, D, dtype=torch.float32, device=o_parts.device)
    if lse is None:
        lse = torch.empty(R, dtype=torch.float32, device=o_parts.device)
    st = library().kvq_merge(_p(o_parts), _p(lse_parts), R, S, D, _p(out), _p(lse), _stream())
    _lib.check(st, "kvq_merge")
    return out, lse


# ---------------------------------------------------------------------------
# Operators over rows of new tokens.  A serving step makes several of these
# calls per layer, so the wrappers test what has to hold in a few expressions
# and work out what to say only when something does not.
# ---------------------------------------------------------------------------

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}
_HALF = (torch.bfloat16, torch.float16)
_STATUS = (torch.int32, torch.uint32)
_SCALES = (torch.float16, torch.int16, torch.uint16)


def _rows(t: torch.Tensor, name: str, dtypes, tokens=None, heads=None, dim=None) -> Rows:
    """A [tokens, heads, head_dim] tensor as the library reads it where it lies:
    channels contiguous, token and head strides multiples of 16 bytes."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3 and t.dtype in dtypes:
        n, h, d = t.shape
        if (tokens is None or n == tokens) and (heads is None or h == heads) and (dim is None or d == dim) and \
                not (t.requires_grad and torch.is_grad_enabled()) and not _has_tangent(t):
            st, sh, sc = t.stride()
            if n == 1:
                st = h * d  # a single token's (head's) stride is free
            if h == 1:
                sh = d
            ptr = t.data_ptr()
            unit = 3 if t.dtype is torch.float32 else 7
            if sc == 1 and st >= d and sh >= d and not (st | sh) & unit and not ptr & 15:
                return Rows(ptr, st, sh)
            if n == 0 or h == 0 or d == 0:
                return Rows(None, 0, 0)
    raise ValueError(_why_not_rows(t, name, dtypes, tokens, heads, dim))


def _has_tangent(t: torch.Tensor) -> bool:
    # (no level of forward-mode differentiation entered, as nearly always: nothing to unpack)
    return getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(t).tangent is not None


def _why_not_rows(t, name, dtypes, tokens, heads, dim) -> str:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return f"{name} must be a CUDA tensor"
    if t.dtype not in dtypes:
        return f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}"
    if t.dim() != 3:
        return f"{name} must be [tokens, heads, head_dim], got {t.dim()} dimensions"
    for what, got, want in (("tokens", t.shape[0], tokens), ("heads", t.shape[1], heads), ("channels", t.shape[2], dim)):
        if want is not None and got != want:
            return f"{name} must have {want} {what}, got {got}"
    if t.requires_grad and torch.is_grad_enabled():
        return f"{name} requires a gradient: this operator has no backward pass (use torch.no_grad())"
    if _has_tangent(t):
        return f"{name} has a tangent: this operator has no derivative (unpack it first)"
    return (f"{name} must have contiguous channels, token and head strides that are multiples of 16 bytes (at least "
            f"head_dim elements) and a 16-byte aligned start; got strides {tuple(t.stride())}")


def _ptr(t, name: str, dtypes, numel: int, device: int):
    """Address of an optional contiguous tensor of that many elements on that device."""
    if t is None:
        return None
    if t.dtype in dtypes and t.numel() == numel and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtypes, numel)
    raise ValueError(f"{name} is on {t.device}, the rows are on cuda:{device}")


def _starts(cu_seqlens, device: int):
    """(batch, address) of the row offsets."""
    if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() == 1:
        n = cu_seqlens.numel()
        if n >= 2:
            return n - 1, _ptr(cu_seqlens, "cu_seqlens", (torch.int32,), n, device)
    raise ValueError("cu_seqlens must be int32 [batch + 1]")


def _blocks_per_sequence(batch: int, page_table, max_blocks, device: int, what: str):
    """(max_blocks, page table address)."""
    if page_table is not None:
        if page_table.dim() != 2 or page_table.shape[0] != batch:
            raise ValueError("page_table must be int32 [batch, max_blocks]")
        mb = page_table.shape[1]
        return mb, _ptr(page_table, "page_table", (torch.int32,), batch * mb, device)
    if max_blocks is None:
        raise ValueError(f"{what} needs page_table, or max_blocks for a contiguous cache")
    return int(max_blocks), None


def _cache_ptrs(desc: CacheDesc, name: str, cache, device: int):
    codes, scale, zero = cache
    blocks = desc.num_pages * desc.num_kv_heads * BLOCK_TOKENS * desc.head_dim
    n = blocks // (desc.group_size or 128)
    return (_ptr(codes, name + " codes", (torch.uint8,), blocks * desc.bits // 8, device),
            _ptr(scale, name + " scale", _SCALES, n, device), _ptr(zero, name + " zero", _SCALES, n, device))


def _apart(at: int, size: int, name: str, rows, tokens: int, heads, dim: int) -> None:
    """Refuses an output over the memory of rows that other CTAs may still read."""
    for r, h in zip(rows, heads):
        read = ((tokens - 1) * r.stride_token + (h - 1) * r.stride_head + dim) * 2
        if tokens and r.data and at < r.data + read and r.data < at + size:
            raise ValueError(f"{name} overlaps the rows that are read")


def _outputs(q: torch.Tensor, T: int, Hq: int, D: int, out, lse, return_lse: bool, device: int, rows, heads):
    """(out, lse, their addresses); what is not given is made."""
    if out is None:
        out = q.new_empty(T, Hq, D)
        po = out.data_ptr()
    else:
        po = _ptr(out, "out", (q.dtype,), T * Hq * D, device)
        _apart(po, T * Hq * D * 2, "out", rows, T, heads, D)
    if lse is None:
        if not return_lse:
            return out, None, po, None
        lse = q.new_empty(T, Hq, dtype=torch.float32)
        return out, lse, po, lse.data_ptr()
    pl = _ptr(lse, "lse", (torch.float32,), T * Hq, device)
    _apart(pl, T * Hq * 4, "lse", rows, T, heads, D)
    if T and po < pl + T * Hq * 4 and pl < po + T * Hq * D * 2:
        raise ValueError("lse overlaps out")
    return out, lse, po, pl


def _launch(device: int, what: str, fn, *args):
    """fn(*args, stream) with the rows' device current, on its current stream."""
    if torch.cuda.current_device() == device:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if st != _lib.KVQ_OK:
        _lib.check(st, what)


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True,
                sm_scale: float = 0.0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                return_lse: bool = False, dev_status: Optional[torch.Tensor] = None, flags: int = 0):
    """Attention over whole prompts, packed: q [T, Hq, D], k and v [T, Hkv, D]
    (bf16 or fp16, strided slices of a fused projection as they are), sequence b
    in rows [cu_seqlens[b], cu_seqlens[b + 1]).  Returns out [T, Hq, D] in q's
    type, and with return_lse (or an lse buffer) also lse fp32 [T, Hq].  Rows
    outside every sequence are left as they were.  Inference only."""
    qr = _rows(q, "q", _HALF)
    T, Hq, D = q.shape
    dt = (q.dtype,)
    kr = _rows(k, "k", dt, T, None, D)
    Hkv = k.shape[1]
    vr = _rows(v, "v", dt, T, Hkv, D)
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"q, k and v are on {q.device}, {k.device} and {v.device}")
    B, pcu = _starts(cu_seqlens, dev)
    out, lse, po, pl = _outputs(q, T, Hq, D, out, lse, return_lse, dev, (qr, kr, vr), (Hq, Hkv, Hkv))
    d = PromptDesc(_DTYPES[q.dtype], D, Hq, Hkv, B, T, 1 if causal else 0, sm_scale, flags)
    _launch(dev, "kvq_prompt_attn", library().kvq_prompt_attn, ctypes.byref(d), ctypes.byref(qr), ctypes.byref(kr),
            ctypes.byref(vr), pcu, po, pl, _ptr(dev_status, "dev_status", _STATUS, 1, dev))
    return out if lse is None else (out, lse)


def _windows_apart(kw, kwo, vw, vwo, size: int, kr: Rows, vr: Rows, T: int, H: int, D: int, element: int) -> None:
    """Refuses windows (of `size` bytes each) that are written over memory that
    the call reads or writes elsewhere."""
    if kw and vw and (abs(kwo - vw) < size or abs(kwo - vwo) < size or abs(vwo - kw) < size):
        raise ValueError("k_window and v_window share the same memory")
    if kw and 0 < abs(kwo - kw) < size or vw and 0 < abs(vwo - vw) < size:
        raise ValueError("a window's output overlaps it in part")
    k, v = kr.data, vr.data
    if T and k and v:
        k_end = k + ((T - 1) * kr.stride_token + (H - 1) * kr.stride_head + D) * element
        v_end = v + ((T - 1) * vr.stride_token + (H - 1) * vr.stride_head + D) * element
        for o in (kwo, vwo):
            if o and (o < k_end and k < o + size or o < v_end and v < o + size):
                raise ValueError("a window overlaps the rows that are read")


def append_chunk(desc: CacheDesc, k_new: torch.Tensor, v_new: torch.Tensor, cu_seqlens: torch.Tensor,
                 seq_lens: torch.Tensor, k_cache, v_cache, k_window: Optional[torch.Tensor] = None,
                 v_window: Optional[torch.Tensor] = None, page_table: Optional[torch.Tensor] = None,
                 max_blocks: Optional[int] = None, k_window_out: Optional[torch.Tensor] = None,
                 v_window_out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None):
    """Append a ragged chunk of new tokens to the packed K and V caches: rows
    [cu_seqlens[b], cu_seqlens[b + 1]) of k_new and v_new [T, Hkv, head_dim]
    (bf16, fp16 or fp32, strided) go to positions seq_lens[b], ... of sequence
    b.  The windows (fp32 [B, Hkv, 128, head_dim]) hold the raw rows of each
    sequence's partial last block, as for append; they are updated in place
    unless *_window_out is given.  A token-wise cache may do without, but append
    must not follow inside a block written so: it quantises the whole block from
    its window (chunks of one row do not).  The caller advances seq_lens
    afterwards.  Returns (k_cache, v_cache)."""
    H, D = desc.num_kv_heads, desc.head_dim
    kr = _rows(k_new, "k_new", _DTYPES, None, H, D)
    T = k_new.shape[0]
    vr = _rows(v_new, "v_new", (k_new.dtype,), T, H, D)
    dev = k_new.get_device()
    if v_new.get_device() != dev:
        raise ValueError(f"k_new is on {k_new.device}, v_new on {v_new.device}")
    B, pcu = _starts(cu_seqlens, dev)
    mb, pt = _blocks_per_sequence(B, page_table, max_blocks, dev, "append_chunk")
    if seq_lens is None:
        raise ValueError("seq_lens must be int32 [batch]")
    windows, size = [], B * H * BLOCK_TOKENS * D
    for name, w, o, scheme in (("k_window", k_window, k_window_out, desc.k_scheme),
                               ("v_window", v_window, v_window_out, desc.v_scheme)):
        if w is None:
            if o is not None or scheme == CHANNELWISE:
                raise ValueError(f"{name} is required (a channel-wise group runs along the block's tokens)")
            windows += [None, None]
            continue
        pw = _ptr(w, name, (torch.float32,), size, dev)
        windows += [pw, pw if o is None else _ptr(o, name + "_out", (torch.float32,), size, dev)]
    kw, kwo, vw, vwo = windows
    if kw or vw:
        _windows_apart(kw, kwo, vw, vwo, size * 4, kr, vr, T, H, D, k_new.element_size())
    _launch(dev, "kvq_append_chunk", library().kvq_append_chunk, ctypes.byref(desc), _DTYPES[k_new.dtype],
            ctypes.byref(kr), ctypes.byref(vr), B, T, pcu, _ptr(seq_lens, "seq_lens", (torch.int32,), B, dev), pt, mb,
            kw, vw, kwo, vwo, *_cache_ptrs(desc, "k_cache", k_cache, dev), *_cache_ptrs(desc, "v_cache", v_cache, dev),
            _ptr(dev_status, "dev_status", _STATUS, 1, dev))
    return k_cache, v_cache


def chunk_workspace_size(desc: CacheDesc, batch: int, total_tokens: int, num_q_heads: int, max_blocks: int) -> int:
    """Workspace bytes of a chunk_attn call with these sizes (the same for every
    batch, number of tokens and heads of a cache geometry)."""
    return _workspace_bytes(ChunkDesc(desc, _lib.BF16, batch, total_tokens, num_q_heads, max_blocks, 1, 0.0, 0))


def _workspace_bytes(d: ChunkDesc) -> int:
    n = ctypes.c_size_t()
    _lib.check(library().kvq_chunk_workspace_size(ctypes.byref(d), ctypes.byref(n)), "kvq_chunk_workspace_size")
    return n.value


def chunk_attn(desc: CacheDesc, q: torch.Tensor, k_cache, v_cache, cu_seqlens: torch.Tensor, seq_lens: torch.Tensor,
               page_table: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None, causal: bool = True,
               sm_scale: float = 0.0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               return_lse: bool = False, workspace: Optional[torch.Tensor] = None,
               dev_status: Optional[torch.Tensor] = None, flags: int = 0):
    """Attention of a ragged chunk of new tokens over the packed cache that
    already holds them: q [T, Hq, D] (bf16 or fp16, strided), sequence b in rows
    [cu_seqlens[b], cu_seqlens[b + 1]), the last of them at position
    seq_lens[b] - 1.  Returns out [T, Hq, D] in q's type, and with return_lse
    (or an lse buffer) also lse fp32 [T, Hq].  Inference only."""
    D = desc.head_dim
    qr = _rows(q, "q", _HALF, None, None, D)
    T, Hq, _ = q.shape
    dev = q.get_device()
    B, pcu = _starts(cu_seqlens, dev)
    mb, pt = _blocks_per_sequence(B, page_table, max_blocks, dev, "chunk_attn")
    if seq_lens is None:
        raise ValueError("seq_lens must be int32 [batch]")
    pk, pv = _cache_ptrs(desc, "k_cache", k_cache, dev), _cache_ptrs(desc, "v_cache", v_cache, dev)
    out, lse, po, pl = _outputs(q, T, Hq, D, out, lse, return_lse, dev, (qr,), (Hq,))
    d = ChunkDesc(desc, _DTYPES[q.dtype], B, T, Hq, mb, 1 if causal else 0, sm_scale, flags)
    if workspace is None:
        size = _workspace_bytes(d)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        pw = workspace.data_ptr()
    else:
        size = workspace.numel()
        pw = _ptr(workspace, "workspace", (torch.uint8,), size, dev)
        if T and qr.data:
            read = ((T - 1) * qr.stride_token + (Hq - 1) * qr.stride_head + D) * 2
            for p, n in (po, T * Hq * D * 2), (pl or 0, T * Hq * 4), (qr.data, read):
                # (of a longer workspace, the first bytes are used)
                if p < pw + size and pw < p + n and p < pw + _workspace_bytes(d):
                    raise ValueError("workspace overlaps q, out or lse")
    _launch(dev, "kvq_chunk_attn", library().kvq_chunk_attn, ctypes.byref(d), ctypes.byref(qr), *pk, *pv, pcu,
            _ptr(seq_lens, "seq_lens", (torch.int32,), B, dev), pt, po, pl, pw, size,
            _ptr(dev_status, "dev_status", _STATUS, 1, dev))
    return out if lse is None else (out, lse)

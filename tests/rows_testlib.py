"""Shared helpers for the tests of the operators over rows of new tokens: the
definitions in 64 bits and elementwise error bounds derived from the roundings
that the operators document."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import kvq_oracle as orc

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # relative half step of a rounding
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def starts(lens, first=0):
    return torch.tensor(np.cumsum([first] + list(lens)), dtype=torch.int32)


def attend64(q, k, v, before, causal, scale, u_p):
    """q [n, H, D], k and v [L, Hkv, D] (any floating type, one device); query i
    at position before + i.  Returns out and lse in 64 bits and the bound of
    out's error before its final rounding, elementwise:

      * the probabilities are rounded (u_p relative) and may lose 2^-32 each
        where they are 16-bit floating point with 5 exponent bits;
      * a score is a sum of D products in fp32 in any order, each addition off
        by at most 2^-23 of the sum of magnitudes, so a weight is off by
        2 E_S relative, E_S = scale D 2^-23 max_t |q| . |k_t|;
      * exp2, the normaliser's sum and the division: 2^-14 relative for up to
        2^17 tokens (128 serial additions a tile, one per tile, one per part).
    """
    q, k, v = q.double(), k.double(), v.double()
    n, H, D = q.shape
    L, Hkv, _ = k.shape
    rep = H // Hkv
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    ltol = torch.zeros_like(lse)
    at = before + torch.arange(n, device=q.device)
    for h in range(H):
        kh, vh, qh = k[:, h // rep], v[:, h // rep], q[:, h]
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            last = int(at[i1 - 1]) if causal else L - 1
            if last < 0 or L == 0:
                continue
            kk, vv = kh[:last + 1], vh[:last + 1]  # later tokens are seen by none of these rows
            s = scale * qh[i0:i1] @ kk.T
            mag = scale * qh[i0:i1].abs() @ kk.abs().T
            if causal:
                hide = torch.arange(len(kk), device=q.device)[None, :] > at[i0:i1, None]
                s = s.masked_fill(hide, -math.inf)
                mag = mag.masked_fill(hide, 0.0)
            some = (s.amax(1) > -math.inf)
            w = torch.softmax(torch.where(some[:, None], s, torch.zeros_like(s)), 1)
            e_s = D * 2.0 ** -23 * mag.amax(1)[:, None]
            # a hidden token's weight is zero whatever its value
            seen = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv))
            o = w @ seen
            a = w @ seen.abs()
            out[i0:i1, h] = torch.where(some[:, None], o, torch.zeros_like(o))
            tol[i0:i1, h] = (u_p + 2 * e_s + 2.0 ** -14) * a + len(kk) * 2.0 ** -32 * seen.abs().amax()
            lse[i0:i1, h] = torch.logsumexp(s, 1)
            ltol[i0:i1, h] = e_s[:, 0] + 2.0 ** -14
    return out, lse, tol, ltol


def assert_rows_close(got, ref, tol, dtype, what=""):
    """got (16-bit) against ref (64 bits): tol, plus got's own rounding."""
    u = HALF_STEP[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half of the smallest fp16 step
    bound = tol * (1 + u) + u * ref.abs() + tiny
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: off by {err.max().item():.3e}, {worst:.3e} over the bound"


def assert_lse_close(got, ref, ltol, what=""):
    """fp32 lse against 64 bits: ltol plus its own rounding."""
    empty = torch.isinf(ref)
    assert torch.equal(torch.isinf(got) & (got < 0), empty), f"{what}: empty rows"
    err = (got.double() - ref).abs()[~empty]
    bound = (ltol + ref.abs() * 2.0 ** -22)[~empty]
    assert (err <= bound).all(), f"{what}: lse off by {err.max().item():.3e}"


def cache_values(cache, lens, bits, which, scheme, page_table, head_dim, rounded=True):
    """Values of a packed cache (CPU arrays of a K or V cache) as float64
    [B, L, Hkv, D], from the oracle's reading; rounded: to fp16, once, as the
    operands of chunk attention are."""
    codes, s, z = cache
    L = max(1, int(max(lens)))
    pt = None if page_table is None else page_table.numpy()
    c, ss, zz = orc.unpack_cache(codes.numpy(), s.numpy(), z.numpy(), lens, bits, which, L, pt)
    x = orc.dequantize(c, ss, zz, lens, scheme)
    if rounded:
        x = x.astype(np.float16).astype(np.float64)
    return torch.from_numpy(x).transpose(1, 2)

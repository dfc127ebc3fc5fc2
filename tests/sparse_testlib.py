"""Shared helpers for the tests of decode steps over part of a cache: caches of
random content, the selection and the attention by their definitions in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import torch

import kvq_synth as synth
from oracle import kvq_oracle as orc


class Cache:
    """Packed K and V caches of ragged sequences, on the GPU and as values."""

    def __init__(self, bits, schemes, hkv, lens, dim=128, group=128, paged=True, seed=1, loud=True):
        import bit_quantized_kv_decode_gb300 as kvq
        self.bits, self.schemes, self.hkv, self.dim, self.group, self.lengths = bits, schemes, hkv, dim, group, list(lens)
        B = len(lens)
        self.wide = max(1, max((n + 127) // 128 for n in lens))
        t = torch.tensor(lens, dtype=torch.int32)
        if paged:
            self.table_host, pages = synth.page_table_for(t, seed, self.wide)
            self.table = self.table_host.cuda()
        else:
            self.table_host, self.table, pages = None, None, B * self.wide
        self.pages = max(1, pages)
        self.desc = kvq.cache_desc(bits, *schemes, hkv, self.pages, head_dim=dim, group=group)
        g = torch.Generator(device="cuda").manual_seed(seed)
        scale = 1.0 + (4.0 * torch.randn(hkv, 1, dim, generator=g, device="cuda").abs() if loud else 0.0)
        L = max(1, max(lens))
        x = torch.randn(B, hkv, L, dim, generator=g, device="cuda")
        x += 0.7 * torch.randn(B, hkv, self.wide, dim, generator=g, device="cuda").repeat_interleave(128, 2)[:, :, :L]
        self.lens = t.cuda()
        self.k = kvq.pack(self.desc, 0, x * scale, self.lens, self.table, self.wide)
        x = torch.randn(B, hkv, L, dim, generator=g, device="cuda")
        self.v = kvq.pack(self.desc, 1, x, self.lens, self.table, self.wide)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.generator = g

    def queries(self, per):
        return torch.randn(len(self.lengths), per * self.hkv, self.dim, generator=self.generator, device="cuda").to(torch.bfloat16)

    def values(self, which):
        """float64 [B, L, Hkv, D], by the oracle's reading of the packed arrays."""
        codes, s, z = (t.cpu().numpy() for t in (self.k, self.v)[which])
        L = max(1, max(self.lengths))
        table = None if self.table_host is None else self.table_host.numpy()
        c, ss, zz = orc.unpack_cache(codes, s, z, self.lengths, self.bits, which, L, table)
        return torch.from_numpy(orc.dequantize(c, ss, zz, self.lengths, self.schemes[which])).transpose(1, 2)

    def page(self, b, j):
        return int(self.table_host[b, j]) if self.table_host is not None else b * self.wide + j


def scores64(cache, q):
    """Block scores by the definition, a list of float64 [Hkv, blocks] per sequence; -inf where not a number."""
    s_all, z_all = (t.double().cpu().numpy() for t in cache.k[1:])
    q = q.double().cpu().numpy()
    groups, most = 128 // cache.group, 2 ** cache.bits - 1
    found = []
    for b, n in enumerate(cache.lengths):
        nb = (n + 127) // 128
        score = np.full((cache.hkv, nb), -np.inf)
        for j in range(nb):
            page = cache.page(b, j)
            s, z = (t[page].reshape(cache.hkv, groups, cache.dim) for t in (s_all, z_all))
            for h in range(cache.hkv):
                per = q.shape[1] // cache.hkv
                for g in range(groups):
                    if j * 128 + g * cache.group >= n:
                        continue
                    lo, hi = z[h, g], z[h, g] + most * s[h, g]
                    with np.errstate(invalid="ignore"):
                        total = sum(np.maximum(x * lo, x * hi).sum() for x in q[b, h * per:(h + 1) * per])
                    if total > score[h, j]:
                        score[h, j] = total
        found.append(score)
    return found


def select64(score, budget, first, last):
    """Ascending block numbers of one list."""
    n = len(score)
    if n <= budget:
        return list(range(n))
    forced = set(range(first)) | set(range(n - last, n))
    rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-score[j], j))
    return sorted(forced | set(rest[:budget - len(forced)]))


def attend_lists64(cache, q, lists, scale=None):
    """out [B, Hq, D] and lse [B, Hq] in 64 bits; lists[b][h]: block numbers."""
    k, v = cache.values(0), cache.values(1)
    q = q.double().cpu()
    B, Hq, D = q.shape
    per = Hq // cache.hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, lse = torch.zeros(B, Hq, D, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(cache.lengths):
        for h in range(cache.hkv):
            at = [t for j in lists[b][h] for t in range(j * 128, min(n, j * 128 + 128))]
            if not at:
                continue
            heads = slice(h * per, (h + 1) * per)
            s = scale * q[b, heads] @ k[b, at, h].T
            out[b, heads] = torch.softmax(s, -1) @ v[b, at, h]
            lse[b, heads] = torch.logsumexp(s, -1)
    return out, lse


def as_lists(lists, list_len, hkv):
    blocks = torch.full((len(lists), hkv, list_len), -1, dtype=torch.int32)
    counts = torch.zeros(len(lists), hkv, dtype=torch.int32)
    for b, of in enumerate(lists):
        for h, x in enumerate(of):
            blocks[b, h, :len(x)] = torch.tensor(x, dtype=torch.int32)
            counts[b, h] = len(x)
    return blocks.cuda(), counts.cuda()


def assert_sparse_close(out, lse, ref, ref_lse, scale_factor=1.0):
    """The tolerance of the E4M3 operands (3e-2 of the result's rms, 1e-2 of lse at the default scale) and the output's
    rounding to bf16 (2^-8 of it)."""
    rms = float((ref ** 2).mean().sqrt()) or 1.0
    err = (out.double().cpu() - ref).abs()
    assert (err <= 3e-2 * rms + 2.0 ** -8 * (ref.abs() + 3e-2 * rms)).all(), f"off by {err.max().item() / rms:.3e} rms"
    if lse is not None:
        empty = torch.isinf(ref_lse)
        assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), empty)
        worst = (lse.double().cpu() - ref_lse).abs()[~empty]
        assert (worst <= 1e-2 * max(1.0, scale_factor)).all(), f"lse off by {worst.max().item():.3e}"

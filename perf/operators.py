"""The cases on which the prompt-side operators are measured: attention over
whole prompts, quantising chunks of new tokens into the cache, and attention
of chunks of new tokens over the quantised, paged cache.

`run` computes either the plain form (elementary torch operations in 32 bits)
or, with `own` set, calls the library as a serving program does.  Sequence
lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one short prompt: an interactive request, where latency counts
        {"name": "prompt_one_short", "op": "prompt", "dtype": "bf16", "batch": 1, "tokens": 256, "heads": 32,
         "kv_heads": 8, "dim": 128, "ragged": False, "causal": True, "fused": True, "mix": 1},
        # a packed batch of prompts of very different lengths, as a scheduler admits them
        {"name": "prompt_packed_ragged", "op": "prompt", "dtype": "bf16", "batch": 24, "tokens": 12289, "heads": 32,
         "kv_heads": 8, "dim": 128, "ragged": True, "causal": True, "fused": True, "mix": 2},
        # one long document
        {"name": "prompt_16k", "op": "prompt", "dtype": "bf16", "batch": 1, "tokens": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "ragged": False, "causal": True, "fused": False, "mix": 3},
        # the large head dim, in the other 16-bit type, two prompts of odd length
        {"name": "prompt_d256_fp16", "op": "prompt", "dtype": "fp16", "batch": 2, "tokens": 6001, "heads": 16,
         "kv_heads": 8, "dim": 256, "ragged": True, "causal": True, "fused": False, "mix": 4},
        # one decode step of a running batch written to the cache (the window re-quantised)
        {"name": "append_step", "op": "append", "dtype": "bf16", "batch": 128, "chunk": 1, "cached": 4096, "kv_heads": 8,
         "dim": 128, "group": 128, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True, "ragged": True, "mix": 5},
        # a long prompt written in one call
        {"name": "append_prompt", "op": "append", "dtype": "bf16", "batch": 4, "chunk": 16384, "cached": 0, "kv_heads": 8,
         "dim": 128, "group": 128, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True, "ragged": False, "mix": 6},
        # chunks of several hundred tokens that start and end inside blocks, 2 bits, small groups
        {"name": "append_ragged_int2", "op": "append", "dtype": "fp16", "batch": 32, "chunk": 777, "cached": 2000,
         "kv_heads": 8, "dim": 64, "group": 32, "bits": 2, "k_scheme": 1, "v_scheme": 1, "paged": True, "ragged": True,
         "mix": 7},
        # four drafted tokens of each of 8 sequences checked at once (the 8 x 4K 2-bit workload's cache)
        {"name": "chunk_drafts_int2", "op": "chunk", "dtype": "bf16", "batch": 8, "chunk": 4, "cached": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "group": 128, "bits": 2, "k_scheme": 1, "v_scheme": 0, "paged": False,
         "ragged": False, "mix": 8},
        # the paged ragged workload (lengths log-uniform up to 128K), a few tokens of each sequence
        {"name": "chunk_paged_ragged_int2", "op": "chunk", "dtype": "bf16", "batch": 64, "chunk": 8, "cached": 131072,
         "heads": 32, "kv_heads": 8, "dim": 128, "group": 128, "bits": 2, "k_scheme": 1, "v_scheme": 0, "paged": True,
         "ragged": True, "mix": 9},
        # one step of a chunked prompt: 512 tokens behind 32K cached ones, 4 bits
        {"name": "chunk_512_at_32k", "op": "chunk", "dtype": "bf16", "batch": 1, "chunk": 512, "cached": 32768,
         "heads": 32, "kv_heads": 8, "dim": 128, "group": 128, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True,
         "ragged": False, "mix": 10},
        # several chunked prompts in one call
        {"name": "chunk_4x2k_at_8k", "op": "chunk", "dtype": "bf16", "batch": 4, "chunk": 2048, "cached": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "group": 128, "bits": 4, "k_scheme": 0, "v_scheme": 0, "paged": True,
         "ragged": False, "mix": 11},
        # the head-dim-256, groups-of-64 workload's cache, a few tokens of each of 32 sequences
        {"name": "chunk_d256_g64", "op": "chunk", "dtype": "bf16", "batch": 32, "chunk": 5, "cached": 8000, "heads": 32,
         "kv_heads": 8, "dim": 256, "group": 64, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True, "ragged": True,
         "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prompt", "append", "chunk"])
    dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    kv_heads = rng.choice([1, 2, 4, 8])
    per = rng.choice([1, 2, 4, 8] if op == "chunk" else [1, 2, 3, 4, 7, 8])
    if kv_heads * per > 32:
        kv_heads = 32 // per
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "kv_heads": kv_heads, "dim": dim, "ragged": rng.random() < 0.7,
            "mix": rng.randrange(1 << 30)}
    if op == "prompt":
        tokens = _log(rng, 32, 8192 if dim == 256 else 16384)
        case |= {"batch": min(_log(rng, 1, 32), tokens), "tokens": tokens, "heads": kv_heads * per,
                 "causal": rng.random() < 0.85, "fused": rng.random() < 0.5}
        return case
    case |= {"group": group, "bits": rng.choice([2, 4]), "k_scheme": rng.choice([0, 1]), "v_scheme": rng.choice([0, 1]),
             "paged": rng.random() < 0.7, "batch": _log(rng, 1, 128 if op == "append" else 64)}
    if op == "append":
        case |= {"dtype": rng.choice(["bf16", "fp16", "fp32"]), "chunk": _log(rng, 1, max(1, 65536 // case["batch"])),
                 "cached": _log(rng, 1, 4096)}
        return case
    chunk = _log(rng, 1, min(2048, 8192 // case["batch"]))
    most = min(131072, (1 << 40) // (case["batch"] * chunk * kv_heads * per * dim), (1 << 31) // (case["batch"] * kv_heads * dim))
    case |= {"heads": kv_heads * per, "chunk": chunk, "cached": _log(rng, 1, most)}
    return case


# ------------------------------------------------------------------ lengths


def _lengths(case):
    """(new tokens, tokens cached before) of each sequence."""
    rng = random.Random(case["mix"])
    B, ragged = case["batch"], case["ragged"]
    if case["op"] == "prompt":
        T = case["tokens"]
        if not ragged:
            return [T // B + (b < T % B) for b in range(B)], [0] * B
        w = [math.exp(rng.uniform(0.0, math.log(32.0))) for _ in range(B)]  # lengths spread over a factor of 32
        n = [max(1, int(T * x / sum(w))) for x in w]
        for b in range(B):  # the total exactly, no prompt below one token
            n[b] = max(1, n[b] + T - sum(n))
            if sum(n) == T:
                break
        return n, [0] * B
    new = [_log(rng, max(1, case["chunk"] // 8), case["chunk"]) if ragged else case["chunk"] for _ in range(B)]
    old = [_log(rng, max(1, case["cached"] // 128), case["cached"]) if ragged else case["cached"] for _ in range(B)]
    return new, old


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _starts(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


# -------------------------------------------- the quantiser and the cache, plainly


def _half_toward(x, up):
    """fp32 -> fp16 rounded up (or down)."""
    h = x.to(torch.float16)
    over = h.float() < x if up else h.float() > x
    bits = h.view(torch.int16).int()
    away = (bits >= 0) == up  # the magnitude grows
    moved = torch.where(h == 0, torch.full_like(bits, 1 if up else -32767), torch.where(away, bits + 1, bits - 1))
    return torch.where(over, moved, bits).to(torch.int16).view(torch.float16)


def _quantise(x, valid, bits, scheme, group):
    """Blocks x [N, H, 128, D] with `valid` [N] tokens: codes uint8 [N, H, 128, D]
    and s, z fp16 [N, H, 128 * D / group] in the cache's order."""
    N, H, _, D = x.shape
    live = (torch.arange(BLOCK, device=x.device) < valid[:, None]).view(N, 1, BLOCK, 1)
    axis = -1 if scheme == 0 else 3
    shape = (N, H, BLOCK, D // group, group) if scheme == 0 else (N, H, BLOCK // group, group, D)
    g, ok = x.view(shape), live.expand(N, H, BLOCK, D).reshape(shape)
    lo = torch.where(ok, g, math.inf).amin(axis, keepdim=True)
    hi = torch.where(ok, g, -math.inf).amax(axis, keepdim=True)
    some = lo <= hi
    lo, hi = torch.where(some, lo, 0.0), torch.where(some, hi, 0.0)
    z = _half_toward(lo, False)
    wide = hi - z.float()
    most = 2 ** bits - 1
    s = torch.where(wide == 0, 0.0, _half_toward(wide / torch.full_like(wide, most), True))
    flat = (s == 0) | ~ok
    q = torch.round((g - z.float()) / torch.where(flat, 1.0, s.float())).clamp_(0, most)
    q = torch.where(flat, 0.0, q).to(torch.uint8).reshape(N, H, BLOCK, D)
    return q, s.reshape(N, H, -1), z.reshape(N, H, -1)


def _pack(codes, bits, which):
    """codes [N, H, 128 tokens, D] -> packed blocks [N, H, bytes]: rows are tokens (K)
    or channels (V), 16-byte chunks of a row, chunk-major."""
    rows = codes if which == 0 else codes.transpose(2, 3)
    N, H, R, C = rows.shape
    per = 8 // bits
    part = rows.reshape(N, H, R, C // per, per).int()
    weight = torch.tensor([1 << (bits * i) for i in range(per)], dtype=torch.int32, device=codes.device)
    packed = (part * weight).sum(-1).to(torch.uint8)
    return packed.view(N, H, R, -1, 16).transpose(2, 3).reshape(N, H, -1)


def _unpack(blob, bits, which, D):
    """Packed blocks [N, H, bytes] -> codes uint8 [N, H, 128 tokens, D]."""
    N, H, _ = blob.shape
    R, C = (BLOCK, D) if which == 0 else (D, BLOCK)
    rows = blob.view(N, H, -1, R, 16).transpose(2, 3).reshape(N, H, R, -1, 1)
    shift = torch.arange(0, 8, bits, dtype=torch.uint8, device=blob.device)
    codes = ((rows >> shift) & (2 ** bits - 1)).view(N, H, R, C)
    return codes if which == 0 else codes.transpose(2, 3)


def _read(cache, pages, case, which):
    """The values x_hat = s * code + z of the blocks in `pages`, fp32 [H, tokens, D]."""
    D, G = case["dim"], case["group"]
    blob, s, z = (t[pages] for t in cache)
    codes = _unpack(blob, case["bits"], which, D).float()
    N, H = codes.shape[:2]
    if (case["k_scheme"], case["v_scheme"])[which] == 0:
        s, z = (t.float().view(N, H, BLOCK, D // G, 1) for t in (s, z))
        x = (codes.view(N, H, BLOCK, D // G, G) * s + z)
    else:
        s, z = (t.float().view(N, H, BLOCK // G, 1, D) for t in (s, z))
        x = (codes.view(N, H, BLOCK // G, G, D) * s + z)
    return x.view(N, H, BLOCK, D).transpose(0, 1).reshape(H, N * BLOCK, D)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, old = _lengths(case)
    B, T, D, Hkv = len(new), sum(new), case["dim"], case["kv_heads"]
    dtype = DTYPES[case["dtype"]]
    st = {"case": case, "new": new, "old": old,
          "cu": torch.tensor(_starts(new), dtype=torch.int32, device=dev)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # a few channels of K are far larger than the others, as in trained models
    loud = 1.0 + 4.0 * normal(Hkv, D).abs()
    if case["op"] == "prompt":
        Hq = case["heads"]
        qkv = normal(T, Hq + 2 * Hkv, D)
        qkv[:, Hq:Hq + Hkv] *= loud
        qkv = qkv.to(dtype)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not case["fused"]:  # three projections instead of slices of one
            st["q"], st["k"], st["v"] = (st[n].contiguous() for n in "qkv")
        return st

    total = [a + b for a, b in zip(new, old)]
    wide = max(_blocks(n) for n in total)
    if case["paged"]:
        order = torch.randperm(sum(_blocks(n) for n in total), generator=g, device=dev).int()
        table = torch.full((B, wide), -1, dtype=torch.int32, device=dev)
        slot = torch.arange(wide, device=dev)[None, :]
        count = torch.tensor([_blocks(n) for n in total], device=dev)
        table[slot < count[:, None]] = order
        pages, st["table"] = len(order), table
    else:
        table = torch.arange(B * wide, dtype=torch.int32, device=dev).view(B, wide)
        pages, st["table"] = B * wide, None
    st["where"], st["wide"], st["pages"] = table, wide, pages
    G, bits = case["group"], case["bits"]
    nsz = BLOCK * D // G
    for which, name in ((0, "k"), (1, "v")):
        codes = torch.zeros(pages, Hkv, BLOCK * D * bits // 8, dtype=torch.uint8, device=dev)
        s = torch.zeros(pages, Hkv, nsz, dtype=torch.float16, device=dev)
        z = torch.zeros(pages, Hkv, nsz, dtype=torch.float16, device=dev)
        window = torch.zeros(B, Hkv, BLOCK, D, device=dev)
        scheme = case[name + "_scheme"]
        held = old if case["op"] == "append" else total  # tokens that the cache holds before the call
        for b, n in enumerate(held):
            for j0 in range(0, _blocks(n), 256):  # 32K tokens at a time
                nb = min(256, _blocks(n) - j0)
                x = normal(nb, Hkv, BLOCK, D)
                if which == 0:
                    x *= loud[:, None, :]
                x = x.to(torch.bfloat16).float()
                valid = (n - BLOCK * (j0 + torch.arange(nb, device=dev))).clamp(max=BLOCK)
                q, sb, zb = _quantise(x, valid, bits, scheme, G)
                at = table[b, j0:j0 + nb].long()
                codes[at], s[at], z[at] = _pack(q, bits, which), sb, zb
                if n % BLOCK and j0 + nb == _blocks(n):
                    window[b, :, :n % BLOCK] = x[-1, :, :n % BLOCK]
        st[name + "_cache"] = (codes, s, z)
        if case["op"] == "append":
            st[name + "_window"] = window
            st[name + "_window_out"] = torch.zeros_like(window)
            x = normal(T, Hkv, D)
            st[name + "_new"] = (x * loud if which == 0 else x).to(dtype)
    st["lens"] = torch.tensor(old if case["op"] == "append" else total, dtype=torch.int32, device=dev)
    if case["op"] == "chunk":
        st["q"] = normal(T, case["heads"], D).to(dtype)
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        st["desc"] = kvq.cache_desc(bits, case["k_scheme"], case["v_scheme"], Hkv, pages, head_dim=D, group=G)
        st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if case["op"] == "chunk":
            st["workspace"] = torch.empty(kvq.chunk_workspace_size(st["desc"], B, T, case["heads"], wide),
                                          dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return {"prompt": _run_prompt, "append": _run_append, "chunk": _run_chunk}[st["case"]["op"]](st)


def _attend(q, k, v, first, causal, scale):
    """q [n, H, D], k and v [Hkv, L, D], fp32; query i sits at position first + i.
    Returns out [n, H, D] and lse [n, H]."""
    n, H, D = q.shape
    Hkv, L, _ = k.shape
    s = torch.matmul(q.view(n, Hkv, H // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D), k.transpose(1, 2))
    s = s.mul_(scale).view(Hkv, H // Hkv, n, L)
    if causal:
        at = torch.arange(L, device=q.device)[None, :] > first + torch.arange(n, device=q.device)[:, None]
        s.masked_fill_(at, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(Hkv, -1, L), v).view(Hkv, H // Hkv, n, D) / total
    lse = (top + total.log()).view(H, n).transpose(0, 1)
    return out.reshape(H, n, D).transpose(0, 1), lse


def _run_prompt(st):
    case, q, k, v = st["case"], st["q"], st["k"], st["v"]
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        out, lse = kvq.prompt_attn(q, k, v, st["cu"], causal=case["causal"], return_lse=True)
        return {"out": out, "lse": lse}
    cu, outs, lses = _starts(st["new"]), [], []
    for a, e in zip(cu, cu[1:]):
        o, l = _attend(q[a:e].float(), k[a:e].float().transpose(0, 1), v[a:e].float().transpose(0, 1), 0,
                       case["causal"], 1.0 / math.sqrt(case["dim"]))
        outs.append(o)
        lses.append(l)
    return {"out": torch.cat(outs).to(q.dtype), "lse": torch.cat(lses)}


def _run_chunk(st):
    case, q = st["case"], st["q"]
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        out = kvq.chunk_attn(st["desc"], q, st["k_cache"], st["v_cache"], st["cu"], st["lens"], st["table"],
                             max_blocks=st["wide"], workspace=st["workspace"], dev_status=st["status"])
        return {"out": out}
    cu, outs = _starts(st["new"]), []
    for b, (n, o) in enumerate(zip(st["new"], st["old"])):
        at = st["where"][b, :_blocks(n + o)].long()
        k = _read(st["k_cache"], at, case, 0)[:, :n + o]
        v = _read(st["v_cache"], at, case, 1)[:, :n + o]
        outs.append(_attend(q[cu[b]:cu[b + 1]].float(), k, v, o, True, 1.0 / math.sqrt(case["dim"]))[0])
    return {"out": torch.cat(outs).to(q.dtype)}


def _run_append(st):
    case = st["case"]
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        kvq.append_chunk(st["desc"], st["k_new"], st["v_new"], st["cu"], st["lens"], st["k_cache"], st["v_cache"],
                         st["k_window"], st["v_window"], page_table=st["table"], max_blocks=st["wide"],
                         k_window_out=st["k_window_out"], v_window_out=st["v_window_out"], dev_status=st["status"])
    else:
        dev, new, old, cu = st["cu"].device, st["new"], st["old"], _starts(st["new"])
        touched = [(b, j) for b in range(len(new)) for j in range(old[b] // BLOCK, _blocks(old[b] + new[b]))]
        seq, blk = (torch.tensor(c, device=dev) for c in zip(*touched))
        n, o, c = (torch.tensor(x, device=dev)[seq][:, None] for x in (new, old, cu[:-1]))
        at = blk[:, None] * BLOCK + torch.arange(BLOCK, device=dev)[None, :]  # positions [N, 128]
        fresh, kept = ((at >= o) & (at < o + n))[..., None, None], (at < o)[..., None, None]
        valid = (o + n - blk[:, None] * BLOCK).clamp(max=BLOCK)[:, 0]
        page = st["where"][seq, blk].long()
        last = valid < BLOCK  # the partial last blocks: their rows go into the window
        row = torch.arange(BLOCK, device=dev)[None, :] < valid[last][:, None]
        for which, name in ((0, "k"), (1, "v")):
            x = st[name + "_new"][(c + at - o).clamp(0, cu[-1] - 1)].float()  # [N, 128, H, D]
            x = torch.where(fresh, x, torch.where(kept, st[name + "_window"][seq].transpose(1, 2), 0.0))
            x = x.transpose(1, 2).contiguous()
            q, s, z = _quantise(x, valid, case["bits"], case[name + "_scheme"], case["group"])
            codes, scale, zero = st[name + "_cache"]
            codes[page], scale[page], zero[page] = _pack(q, case["bits"], which), s, z
            out = st[name + "_window_out"]
            out[seq[last]] = torch.where(row[:, None, :, None], x[last], out[seq[last]])
    return {name: {"codes": st[name + "_cache"][0], "scale": st[name + "_cache"][1], "zero": st[name + "_cache"][2],
                   "window": st[name + "_window_out"]} for name in "kv"}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    new, old = _lengths(case)
    T, D, Hkv = sum(new), case["dim"], case["kv_heads"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in new)
        return {"bytes": T * D * size * (2 * case["heads"] + 2 * Hkv) + 4 * T * case["heads"],
                "flops": 4 * pairs * case["heads"] * D}
    token = 2 * Hkv * (D * case["bits"] / 8 + 4 * D / case["group"])  # a token's codes, s and z, of K and V
    if case["op"] == "chunk":
        pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
        return {"bytes": (T + sum(old)) * token + 2 * T * D * size * case["heads"],
                "flops": 4 * pairs * case["heads"] * D}
    # the chunk read and its codes written; the window's raw rows of a partial last block written, those of a block
    # that was begun before read where its groups run along the tokens or where it is still the last
    moved, read = T * (2 * Hkv * D * size + token), 0
    for n, o in zip(new, old):
        r, e = o % BLOCK, (o + n) % BLOCK
        same = (o + n) // BLOCK == o // BLOCK
        read += r * sum(same or case[s] == 1 for s in ("k_scheme", "v_scheme")) * Hkv * D * 4
        moved += 2 * e * Hkv * D * 4
        moved += r * sum(case[s] for s in ("k_scheme", "v_scheme")) * token / 2
    return {"bytes": moved + read, "flops": 6 * 2 * T * Hkv * D}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_rows(q, k, v, first, causal, scale):
    """One query head: q [n, D], k, v [L, D] in 64 bits, 2,048 queries at a time."""
    outs, lses = [], []
    for a in range(0, len(q), 2048):
        s = (q[a:a + 2048] * scale) @ k.T
        if causal:
            at = first + a + torch.arange(len(s), device=q.device)
            s = s.where(torch.arange(len(k), device=q.device) <= at[:, None], -math.inf)
        outs.append(torch.softmax(s, -1) @ v)
        lses.append(torch.logsumexp(s, -1))
    return torch.cat(outs), torch.cat(lses)


def _exact_value(cache, page, head, tok, case, which):
    """Values of tokens `tok` (positions in their pages) of one KV head, [n, D], in 64 bits, each
    code fetched by its address in the format's definition."""
    blob, s, z = cache
    D, G, bits = case["dim"], case["group"], case["bits"]
    c = torch.arange(D, device=blob.device)[None, :]
    t, page = tok[:, None], page[:, None]
    row, col, rows = (t, c, BLOCK) if which == 0 else (c, t, D)
    byte = col * bits // 8
    raw = blob[page, head, (byte // 16 * rows + row) * 16 + byte % 16].long()
    code = (raw >> (col * bits % 8)) % 2 ** bits
    entry = t * (D // G) + c // G if (case["k_scheme"], case["v_scheme"])[which] == 0 else (t // G) * D + c
    return s[page, head, entry].double() * code + z[page, head, entry].double()


def exact(case, seed):
    global own
    if work(case)["flops"] > 6e12:
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    dev, new, old, cu = st["cu"].device, st["new"], st["old"], _starts(st["new"])
    D, Hkv = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        return _exact_append(st)
    H = case["heads"]
    out = torch.zeros(cu[-1], H, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(cu[-1], H, dtype=torch.float64, device=dev)
    for b, (n, o) in enumerate(zip(new, old)):
        rows = slice(cu[b], cu[b + 1])
        if case["op"] == "chunk":
            at = torch.arange(n + o, device=dev)
            page = st["where"][b].long()[at // BLOCK]
        for h in range(Hkv):
            if case["op"] == "prompt":
                k, v = st["k"][rows, h].double(), st["v"][rows, h].double()
            else:
                k, v = (_exact_value(st[x + "_cache"], page, h, at % BLOCK, case, w) for w, x in ((0, "k"), (1, "v")))
            for i in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                out[rows, i], lse[rows, i] = _exact_rows(st["q"][rows, i].double(), k, v, o,
                                                         case["op"] == "chunk" or case["causal"], 1.0 / math.sqrt(D))
    return {"out": out, "lse": lse} if case["op"] == "prompt" else {"out": out}


def _exact_append(st):
    """Scales and offsets, block by block; codes are whole numbers and have no value in 64 bits."""
    case, new, old, cu = st["case"], st["new"], st["old"], _starts(st["new"])
    G, D, most = case["group"], case["dim"], 2 ** case["bits"] - 1
    if sum(_blocks(n) + 1 for n in new) > 1200:
        return None
    result = {}
    for name in "kv":
        scale, zero = (t.double() for t in st[name + "_cache"][1:])
        window = st[name + "_window_out"].double()
        for b, (n, o) in enumerate(zip(new, old)):
            for j in range(o // BLOCK, _blocks(o + n)):
                a, e = max(o, j * BLOCK), min(o + n, (j + 1) * BLOCK)
                x = st[name + "_new"][cu[b] + a - o:cu[b] + e - o].double().transpose(0, 1)
                if o > j * BLOCK:
                    x = torch.cat([st[name + "_window"][b, :, :o - j * BLOCK].double(), x], 1)
                H, m, _ = x.shape
                if m < BLOCK:
                    window[b, :, :m] = x
                if case[name + "_scheme"] == 0:
                    parts = [x.reshape(H, m * (D // G), G)]
                else:
                    parts = [x[:, i:i + G].transpose(1, 2) for i in range(0, m, G)]
                s, z = (torch.zeros(H, BLOCK * D // G, dtype=torch.float64, device=x.device) for _ in "sz")
                for i, p in enumerate(parts):
                    lo, hi = p.aminmax(dim=-1)
                    zi = _grid16(lo, torch.floor)
                    si = _grid16(((hi - zi).float().double() / most).float().double(), torch.ceil)
                    s[:, i * D:i * D + zi.shape[1]], z[:, i * D:i * D + zi.shape[1]] = si, zi
                page = int(st["where"][b, j])
                scale[page], zero[page] = s, z
        result[name] = {"codes": None, "scale": scale, "zero": zero, "window": window}
    return result


def _grid16(x, to):
    """x (64 bits) on the grid of 16-bit floating point, by `to` (floor or ceil)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))) - 10)
    return to(x / step) * step

"""The cases on which three operators of a decode step over a long quantised
cache are measured: appending new tokens with the position rotation on the way,
selecting the blocks of the cache that a query may look at, and attention over
the selected blocks alone.

`run` computes either the plain form (elementary torch operations) or, with
`own` set, calls the library as a serving program does.  Sequence lengths
follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    cache = {"kv_heads": 8, "dim": 128, "group": 128, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True}
    return [
        # one decode step of a running batch: every sequence's new token, q rotated beside it
        {"name": "rotary_step", "op": "rotary", "dtype": "bf16", "batch": 128, "chunk": 1, "cached": 4096, **cache,
         "heads": 32, "rotary": 128, "interleaved": False, "k_out": False, "ragged": True, "mix": 1},
        # long prompts written in one call; q and k also go to the prompt's attention
        {"name": "rotary_prompt", "op": "rotary", "dtype": "bf16", "batch": 4, "chunk": 8192, "cached": 0, **cache,
         "heads": 32, "rotary": 128, "interleaved": False, "k_out": True, "ragged": False, "mix": 2},
        # chunks that start and end inside blocks; half of the channels rotated, as neighbouring pairs; K and V alone
        {"name": "rotary_ragged_int2", "op": "rotary", "dtype": "fp16", "batch": 32, "chunk": 777, "cached": 2000,
         "kv_heads": 8, "dim": 64, "group": 32, "bits": 2, "k_scheme": 1, "v_scheme": 1, "paged": True, "heads": 0,
         "rotary": 32, "interleaved": True, "k_out": False, "ragged": True, "mix": 3},
        # a few drafted tokens of 32 sequences on the head-dim-256, groups-of-64 workload's cache
        {"name": "rotary_drafts_d256", "op": "rotary", "dtype": "bf16", "batch": 32, "chunk": 5, "cached": 8000,
         "kv_heads": 8, "dim": 256, "group": 64, "bits": 4, "k_scheme": 1, "v_scheme": 0, "paged": True, "heads": 32,
         "rotary": 256, "interleaved": False, "k_out": False, "ragged": True, "mix": 4},
        # the 8 x 4K 2-bit workload: few short lists, where latency counts
        {"name": "select_8x4k_int2", "op": "select", "batch": 8, "cached": 4096, **cache, "bits": 2, "paged": False,
         "heads": 32, "budget": 8, "first": 1, "last": 1, "ragged": False, "mix": 5},
        # the paged ragged workload (lengths log-uniform up to 128K)
        {"name": "select_paged_ragged", "op": "select", "batch": 64, "cached": 131072, **cache, "bits": 2, "heads": 32,
         "budget": 64, "first": 1, "last": 2, "ragged": True, "mix": 6},
        # the large workload: 128 sequences of 32K
        {"name": "select_128x32k", "op": "select", "batch": 128, "cached": 32768, **cache, "heads": 32, "budget": 32,
         "first": 1, "last": 1, "ragged": False, "mix": 7},
        # one document of a million tokens
        {"name": "select_one_1m", "op": "select", "batch": 1, "cached": 1048571, **cache, "heads": 32, "budget": 256,
         "first": 1, "last": 4, "ragged": False, "mix": 8},
        # attention over what those selections leave
        {"name": "sparse_8x4k_int2", "op": "sparse", "batch": 8, "cached": 4096, **cache, "bits": 2, "paged": False,
         "heads": 32, "budget": 8, "ragged": False, "mix": 9},
        {"name": "sparse_paged_ragged", "op": "sparse", "batch": 64, "cached": 131072, **cache, "bits": 2, "heads": 32,
         "budget": 64, "ragged": True, "mix": 10},
        {"name": "sparse_128x32k", "op": "sparse", "batch": 128, "cached": 32768, **cache, "heads": 32, "budget": 32,
         "ragged": False, "mix": 11},
        {"name": "sparse_one_1m", "op": "sparse", "batch": 1, "cached": 1048571, **cache, "heads": 32, "budget": 256,
         "ragged": False, "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotary", "select", "sparse"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    case = {"op": op, "kv_heads": kv_heads, "dim": dim, "group": rng.choice([g for g in (32, 64, 128) if g <= dim]),
            "bits": rng.choice([2, 4]), "k_scheme": rng.choice([0, 1]), "v_scheme": rng.choice([0, 1]),
            "paged": rng.random() < 0.7, "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 30),
            "heads": kv_heads * rng.choice([1, 2, 4, 8])}
    if op == "rotary":
        rotary = rng.choice([dim, dim, dim // 2, dim // 2 + 16])
        case |= {"dtype": rng.choice(["bf16", "fp16", "fp32"]), "batch": _log(rng, 1, 128), "cached": _log(rng, 1, 4096),
                 "rotary": rotary, "interleaved": rng.random() < 0.4, "k_out": rng.random() < 0.4,
                 "heads": rng.choice([0, case["heads"], case["heads"]])}
        most = 96_000_000 // ((kv_heads + case["heads"] // 2) * dim * case["batch"] * (2 if case["dtype"] == "fp32" else 1))
        return case | {"chunk": _log(rng, 1, max(1, min(8192, most)))}
    batch = _log(rng, 1, 128)
    most = (1 << 30) // (batch * kv_heads * dim)  # tokens of a sequence: no more values than the large workload's
    cached = _log(rng, 512, max(512, min(1 << 20, most)))
    case |= {"batch": batch, "cached": cached, "budget": _log(rng, 4, max(5, min(256, (1 << 22) // (batch * kv_heads * dim))))}
    if op == "select":
        case |= {"k_scheme": 1, "first": rng.randrange(3), "last": rng.randrange(3)}
    return case


# ------------------------------------------------------------------ lengths


def _lengths(case):
    """(new tokens, tokens cached before) of each sequence."""
    rng = random.Random(case["mix"])
    B, ragged = case["batch"], case["ragged"]
    chunk = case.get("chunk", 0)
    new = [_log(rng, max(1, chunk // 8), chunk) if ragged and chunk > 1 else chunk for _ in range(B)]
    old = [_log(rng, max(1, case["cached"] // 128), case["cached"]) if ragged and case["cached"] else case["cached"]
           for _ in range(B)]
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
    """Packed blocks [N, bytes] -> codes uint8 [N, 128 tokens, D]."""
    N = blob.shape[0]
    R, C = (BLOCK, D) if which == 0 else (D, BLOCK)
    rows = blob.view(N, -1, R, 16).transpose(1, 2).reshape(N, R, -1, 1)
    shift = torch.arange(0, 8, bits, dtype=torch.uint8, device=blob.device)
    codes = ((rows >> shift) & (2 ** bits - 1)).view(N, R, C)
    return codes if which == 0 else codes.transpose(1, 2)


def _read(cache, page, head, case, which):
    """The values x_hat = s * code + z of the blocks (page, head) [N], fp32 [N, 128, D]."""
    D, G = case["dim"], case["group"]
    blob, s, z = (t[page, head] for t in cache)
    codes = _unpack(blob, case["bits"], which, D).float().contiguous()
    N = len(codes)
    if (case["k_scheme"], case["v_scheme"])[which] == 0:
        s, z = (t.float().view(N, BLOCK, D // G, 1) for t in (s, z))
        return (codes.view(N, BLOCK, D // G, G) * s + z).view(N, BLOCK, D)
    s, z = (t.float().view(N, BLOCK // G, 1, D) for t in (s, z))
    return (codes.view(N, BLOCK // G, G, D) * s + z).view(N, BLOCK, D)


# ------------------------------------------------------------------ inputs


def _angles(positions, rotary, device):
    """cos, then sin, of the angles of each position, rounded once from 64 bits: fp32 [positions, rotary]."""
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / rotary)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, old = _lengths(case)
    op, B, T, D, H = case["op"], len(new), sum(new), case["dim"], case["kv_heads"]
    total = [a + b for a, b in zip(new, old)]
    wide = max(_blocks(n) for n in total)
    st = {"case": case, "new": new, "old": old, "wide": wide, "status": torch.zeros(1, dtype=torch.int32, device=dev)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # a few channels of K are far larger than the others, as in trained models
    loud = 1.0 + 4.0 * normal(H, D).abs()
    count = torch.tensor([_blocks(n) for n in total], device=dev)
    slot = torch.arange(wide, device=dev)[None, :]
    if case["paged"]:
        pages = sum(_blocks(n) for n in total)
        table = torch.full((B, wide), -1, dtype=torch.int32, device=dev)
        table[slot < count[:, None]] = torch.randperm(pages, generator=g, device=dev).int()
        st["table"] = table
    else:
        pages = B * wide
        table = torch.arange(pages, dtype=torch.int32, device=dev).view(B, wide)
        st["table"] = None
    st["where"], st["pages"] = table, pages
    G, bits = case["group"], case["bits"]
    nsz = BLOCK * D // G
    held = torch.tensor(old, device=dev)
    seq, blk = ((slot * BLOCK < held[:, None])).nonzero().unbind(1)  # the blocks that the cache holds before the call
    valid, page = (held[seq] - blk * BLOCK).clamp(max=BLOCK), table[seq, blk].long()
    step = max(1, (1 << 28) // (H * BLOCK * D))
    for which, name in ((0, "k"), (1, "v")):
        if op == "select" and which == 1:
            break
        codes = torch.zeros(pages, H, BLOCK * D * bits // 8, dtype=torch.uint8, device=dev)
        s = torch.zeros(pages, H, nsz, dtype=torch.float16, device=dev)
        z = torch.zeros(pages, H, nsz, dtype=torch.float16, device=dev)
        window = torch.zeros(B, H, BLOCK, D, device=dev) if op == "rotary" else None
        for i in range(0, len(seq), step):
            at = slice(i, i + step)
            # neighbouring tokens are alike: a block has a mean of its own
            x = normal(len(page[at]), H, BLOCK, D) + 0.7 * normal(len(page[at]), H, 1, D)
            if which == 0:
                x *= loud[:, None, :]
            q, sb, zb = _quantise(x, valid[at], bits, case[name + "_scheme"], G)
            codes[page[at]], s[page[at]], z[page[at]] = _pack(q, bits, which), sb, zb
            if window is not None:
                part = valid[at] < BLOCK
                row = torch.arange(BLOCK, device=dev)[None, :] < valid[at][part][:, None]
                window[seq[at][part]] = torch.where(row[:, None, :, None], x[part], 0.0)
        st[name + "_cache"] = (codes, s, z)
        if op == "rotary":
            st[name + "_window"], st[name + "_window_out"] = window, torch.zeros_like(window)
            x = normal(T, H, D)
            st[name + "_new"] = (x * loud if which == 0 else x).to(DTYPES[case["dtype"]])
    st["lens"] = torch.tensor(old, dtype=torch.int32, device=dev)
    if op == "rotary":
        st["cu"] = torch.tensor(_starts(new), dtype=torch.int32, device=dev)
        st["angles"] = _angles(max(total), case["rotary"], dev)
        st["q"] = normal(T, case["heads"], D).to(DTYPES[case["dtype"]]) if case["heads"] else None
    else:
        st["q"] = normal(B, case["heads"], D).to(torch.bfloat16)
    if op == "sparse":
        # what a selection leaves: the first block, the last, and others in between, in order
        n = count.clamp(max=case["budget"])[:, None].expand(B, H)
        rank = torch.rand(B, H, wide, generator=g, device=dev)
        rank[:, :, 0] = 3.0
        rank.scatter_(2, (count - 1).view(B, 1, 1).expand(B, H, 1), 2.0)
        rank[(slot >= count[:, None])[:, None].expand(B, H, wide)] = -1.0
        k = min(case["budget"], wide)
        at = rank.topk(k, dim=2).indices
        at = torch.where(torch.arange(k, device=dev) < n[..., None], at, wide).sort(2).values
        lists = torch.full((B, H, case["budget"]), -1, dtype=torch.int32, device=dev)
        lists[..., :k] = torch.where(at < wide, at, -1).int()
        st["blocks"], st["counts"] = lists, n.int().contiguous()
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        st["desc"] = kvq.cache_desc(bits, case["k_scheme"], case["v_scheme"], H, pages, head_dim=D, group=G)
        if op == "sparse":
            st["workspace"] = torch.empty(kvq.sparse_workspace_size(st["desc"], B, case["heads"], case["budget"]),
                                          dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return {"rotary": _run_rotary, "select": _run_select, "sparse": _run_sparse}[st["case"]["op"]](st)


def _rotate(x, angle, interleaved):
    """x [T, H, D] in fp32 with the first R channels rotated by angle [T, R] (cos, then sin): every product and
    sum rounded to fp32 by itself, as the codes of the quantised values depend on the last bit."""
    R = angle.shape[1]
    c, s = angle[:, None, :R // 2], angle[:, None, R // 2:]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _run_rotary(st):
    case, k_out = st["case"], None
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        if case["k_out"]:
            k_out = torch.empty_like(st["k_new"])
        q_out = kvq.append_rotary(st["desc"], st["angles"], st["k_new"], st["v_new"], st["cu"], st["lens"], st["k_cache"],
                                  st["v_cache"], st["k_window"], st["v_window"], page_table=st["table"],
                                  max_blocks=st["wide"], k_window_out=st["k_window_out"],
                                  v_window_out=st["v_window_out"], interleaved=case["interleaved"], q=st["q"],
                                  k_out=k_out, dev_status=st["status"])
    else:
        T, dev = len(st["k_new"]), st["cu"].device
        row = torch.arange(T, device=dev)
        seq = torch.searchsorted(st["cu"][1:], row.int(), right=True)
        angle = st["angles"][st["lens"].long()[seq] + row - st["cu"].long()[seq]]
        k = _rotate(st["k_new"].float(), angle, case["interleaved"])
        q_out = _rotate(st["q"].float(), angle, case["interleaved"]).to(st["q"].dtype) if st["q"] is not None else None
        k_out = k.to(st["k_new"].dtype) if case["k_out"] else None
        _store(st, "k", 0, k)
        _store(st, "v", 1, st["v_new"].float())
    result = {name: {"codes": st[name + "_cache"][0], "scale": st[name + "_cache"][1], "zero": st[name + "_cache"][2],
                     "window": st[name + "_window_out"]} for name in "kv"}
    return result | {"q": q_out, "k_rows": k_out}


def _store(st, name, which, rows):
    """rows [T, H, D] (fp32) quantised into the cache behind the tokens that are there."""
    case, dev, new, old, cu = st["case"], st["cu"].device, st["new"], st["old"], _starts(st["new"])
    touched = [(b, j) for b in range(len(new)) for j in range(old[b] // BLOCK, _blocks(old[b] + new[b]))]
    seq, blk = (torch.tensor(c, device=dev) for c in zip(*touched))
    n, o, c = (torch.tensor(x, device=dev)[seq][:, None] for x in (new, old, cu[:-1]))
    at = blk[:, None] * BLOCK + torch.arange(BLOCK, device=dev)[None, :]  # positions [N, 128]
    fresh, kept = ((at >= o) & (at < o + n))[..., None, None], (at < o)[..., None, None]
    valid = (o + n - blk[:, None] * BLOCK).clamp(max=BLOCK)[:, 0]
    page = st["where"][seq, blk].long()
    last = valid < BLOCK  # the partial last blocks: their rows go into the window
    row = torch.arange(BLOCK, device=dev)[None, :] < valid[last][:, None]
    x = rows[(c + at - o).clamp(0, cu[-1] - 1)]  # [N, 128, H, D]
    x = torch.where(fresh, x, torch.where(kept, st[name + "_window"][seq].transpose(1, 2), 0.0))
    x = x.transpose(1, 2).contiguous()
    q, s, z = _quantise(x, valid, case["bits"], case[name + "_scheme"], case["group"])
    codes, scale, zero = st[name + "_cache"]
    codes[page], scale[page], zero[page] = _pack(q, case["bits"], which), s, z
    out = st[name + "_window_out"]
    out[seq[last]] = torch.where(row[:, None, :, None], x[last], out[seq[last]])


def _run_select(st):
    case, q = st["case"], st["q"]
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        blocks, counts = kvq.select_blocks(st["desc"], q, st["k_cache"], st["lens"], case["budget"], first=case["first"],
                                           last=case["last"], page_table=st["table"], max_blocks=st["wide"],
                                           dev_status=st["status"])
        return {"blocks": blocks, "counts": counts}
    # scores in 64 bits: which of two neighbours in rank is taken must not hang on a rounding
    B, H, D, G, wide, k = len(q), case["kv_heads"], case["dim"], case["group"], st["wide"], case["budget"]
    q = q.view(B, H, -1, D).double()
    weight, range_weight = q.sum(2), q.clamp(min=0).sum(2) * (2 ** case["bits"] - 1)  # [B, H, D]
    page = st["where"].long().clamp(min=0)
    s, z = (t[page].view(B, wide, H, BLOCK // G, D).double() for t in st["k_cache"][1:])
    score = (z.mul_(weight[:, None, :, None]).sum(-1) + s.mul_(range_weight[:, None, :, None]).sum(-1))  # [B, wide, H, groups]
    j = torch.arange(wide, device=q.device)
    start = j[:, None] * BLOCK + torch.arange(0, BLOCK, G, device=q.device)  # a group's first token
    score = score.masked_fill((start >= st["lens"][:, None, None])[:, :, None], -math.inf).amax(-1).transpose(1, 2)
    n = ((st["lens"] + BLOCK - 1) // BLOCK)[:, None]
    score = torch.where(((j < case["first"]) | (j >= n - case["last"]))[:, None], math.inf, score)
    score = torch.where((j < n)[:, None], score, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    taken = torch.arange(best.shape[-1], device=q.device) < n[..., None]
    best = torch.where(taken, best, wide).sort(-1).values
    blocks = torch.full((B, H, k), -1, dtype=torch.int32, device=q.device)
    blocks[..., :best.shape[-1]] = torch.where(best < wide, best, -1)
    return {"blocks": blocks, "counts": n.clamp(max=k).expand(B, H).int().contiguous()}


def _run_sparse(st):
    case, q = st["case"], st["q"]
    if own:
        import bit_quantized_kv_decode_gb300 as kvq
        out = kvq.sparse_decode_attn(st["desc"], q, st["k_cache"], st["v_cache"], st["lens"], st["blocks"], st["counts"],
                                     st["table"], max_blocks=st["wide"], workspace=st["workspace"],
                                     dev_status=st["status"])
        return {"out": out}
    B, Hq, D = q.shape
    H, K = case["kv_heads"], case["budget"]
    lists = st["blocks"].long()
    there = torch.arange(K, device=q.device) < st["counts"][..., None]  # [B, H, K]
    page = st["where"].long()[torch.arange(B, device=q.device)[:, None, None], lists.clamp(min=0)].flatten().clamp(min=0)
    head = torch.arange(H, device=q.device)[None, :, None].expand(B, H, K).flatten()
    k = _read(st["k_cache"], page, head, case, 0).view(B, H, K * BLOCK, D)
    s = torch.matmul(q.float().view(B, H, Hq // H, D), k.transpose(2, 3)) / math.sqrt(D)
    del k
    at = lists[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)
    hide = ~(there[..., None] & (at < st["lens"].view(B, 1, 1, 1))).reshape(B, H, 1, K * BLOCK)
    s = s.masked_fill_(hide, -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    v = _read(st["v_cache"], page, head, case, 1).view(B, H, K * BLOCK, D)
    out = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return {"out": out.view(B, Hq, D).to(q.dtype)}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    new, old = _lengths(case)
    D, H, B = case["dim"], case["kv_heads"], len(new)
    token = 2 * H * (D * case["bits"] / 8 + 4 * D / case["group"])  # a token's codes, s and z, of K and V
    if case["op"] == "rotary":
        size, T, Hq = 4 if case["dtype"] == "fp32" else 2, sum(new), case["heads"]
        far = max(n + o for n, o in zip(new, old))
        moved = T * (2 * H * D * size + token + 2 * Hq * D * size + (H * D * size if case["k_out"] else 0))
        moved += min(T, far) * case["rotary"] * 4  # angles of the positions
        for n, o in zip(new, old):
            r, e = o % BLOCK, (o + n) % BLOCK
            same = (o + n) // BLOCK == o // BLOCK
            moved += r * sum(same or case[s] == 1 for s in ("k_scheme", "v_scheme")) * H * D * 4
            moved += 2 * e * H * D * 4
            moved += r * sum(case[s] for s in ("k_scheme", "v_scheme")) * token / 2
        return {"bytes": moved, "flops": T * (6 * 2 * H * D + 3 * (Hq + H) * case["rotary"])}
    n = [_blocks(x) for x in old]
    if case["op"] == "select":
        scored = sum(max(0, x - case["first"] - case["last"]) for x in n if x > case["budget"]) * H
        entries = BLOCK // case["group"] * D  # scales (offsets) of a block
        return {"bytes": scored * entries * 4 + B * case["heads"] * D * 2 + B * H * (case["budget"] + 1) * 4,
                "flops": 4 * scored * entries}
    taken = sum(min(x, case["budget"]) for x in n)
    return {"bytes": taken * BLOCK * token + B * case["heads"] * D * 4 + B * H * (case["budget"] + 1) * 4,
            "flops": 4 * taken * BLOCK * case["heads"] * D}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rotary": _exact_rotary, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](st)


def _exact_turn(x, angle, interleaved):
    """Rows [n, H, D] times the rotation matrix of each token, [n, D, D], in 64 bits."""
    n, _, D = x.shape
    R = angle.shape[1]
    m = torch.eye(D, dtype=torch.float64, device=x.device).repeat(n, 1, 1)
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    c, s = angle[:, :R // 2].double(), angle[:, R // 2:].double()
    m[:, a, a], m[:, b, b], m[:, a, b], m[:, b, a] = c, c, s, -s
    return torch.matmul(x.double(), m)


def _exact_rotary(st):
    """Rotated rows, scales and offsets, block by block; codes are whole numbers and have no value in 64 bits."""
    case, new, old, cu = st["case"], st["new"], st["old"], _starts(st["new"])
    G, D, most = case["group"], case["dim"], 2 ** case["bits"] - 1
    if sum(_blocks(n) + 1 for n in new) > 1200:
        return None
    turned = {}
    for name in ("k_new", "q"):
        if st[name] is None:
            continue
        parts = []
        for b, (n, o) in enumerate(zip(new, old)):
            for i in range(0, n, 2048):
                m = min(2048, n - i)
                parts.append(_exact_turn(st[name][cu[b] + i:cu[b] + i + m], st["angles"][o + i:o + i + m], case["interleaved"]))
        turned[name] = torch.cat(parts)
    rows = {"k": turned["k_new"], "v": st["v_new"].double()}
    result = {}
    for name in "kv":
        scale, zero = (t.double() for t in st[name + "_cache"][1:])
        window = st[name + "_window_out"].double()
        for b, (n, o) in enumerate(zip(new, old)):
            for j in range(o // BLOCK, _blocks(o + n)):
                a, e = max(o, j * BLOCK), min(o + n, (j + 1) * BLOCK)
                x = rows[name][cu[b] + a - o:cu[b] + e - o].transpose(0, 1)
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
                    si = _grid16((hi - zi) / most, torch.ceil)
                    s[:, i * D:i * D + zi.shape[1]], z[:, i * D:i * D + zi.shape[1]] = si, zi
                page = int(st["where"][b, j])
                scale[page], zero[page] = s, z
        result[name] = {"codes": None, "scale": scale, "zero": zero, "window": window}
    return result | {"q": turned.get("q"), "k_rows": turned["k_new"] if case["k_out"] else None}


def _grid16(x, to):
    """x (64 bits) on the grid of 16-bit floating point, by `to` (floor or ceil)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))) - 10)
    return to(x / step) * step


def _exact_select(st):
    """The lists, by the definition: a token group's channel c holds values in [z, z + most * s]; its score is the sum
    over the query heads of the largest q . k with k in that box."""
    case = st["case"]
    B, H, D, G, k = len(st["q"]), case["kv_heads"], case["dim"], case["group"], case["budget"]
    blocks = torch.full((B, H, k), -1, dtype=torch.int64, device=st["q"].device)
    counts = torch.zeros(B, H, dtype=torch.int64, device=st["q"].device)
    for b, length in enumerate(st["old"]):
        n = _blocks(length)
        s, z = (t[st["where"][b, :n].long()].double().view(n, H, BLOCK // G, D) for t in st["k_cache"][1:])
        top = z + (2 ** case["bits"] - 1) * s
        score = torch.zeros(n, H, BLOCK // G, dtype=torch.float64, device=s.device)
        for q in st["q"][b].double().view(H, -1, D).unbind(1):
            score += torch.maximum(q[:, None] * z, q[:, None] * top).sum(-1)
        inside = (n - 1) * BLOCK + torch.arange(0, BLOCK, G, device=s.device) < length
        score[-1] = score[-1].masked_fill(~inside, -math.inf)
        score = score.amax(-1)
        score[:case["first"]] = math.inf
        score[max(0, n - case["last"]):] = math.inf
        best = score.argsort(dim=0, descending=True, stable=True)[:k].sort(0).values
        blocks[b, :, :len(best)] = best.T
        counts[b] = len(best)
    return {"blocks": blocks, "counts": counts}


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


def _exact_sparse(st):
    case, q = st["case"], st["q"].double()
    B, Hq, D = q.shape
    H = case["kv_heads"]
    if work(case)["flops"] > 1e12:
        return None
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    lists, counts = st["blocks"].tolist(), st["counts"].tolist()
    for b, length in enumerate(st["old"]):
        for h in range(H):
            at = torch.tensor(lists[b][h][:counts[b][h]], device=q.device)[:, None] * BLOCK + torch.arange(BLOCK, device=q.device)
            at = at[at < length]
            page = st["where"][b].long()[at // BLOCK]
            k, v = (_exact_value(st[x + "_cache"], page, h, at % BLOCK, case, w) for w, x in ((0, "k"), (1, "v")))
            heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
            out[b, heads] = torch.softmax(q[b, heads] @ k.T / math.sqrt(D), -1) @ v
    return {"out": out}

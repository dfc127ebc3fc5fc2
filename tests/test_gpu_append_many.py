"""Appends of few tokens to many sequences, nearly all of them without any: the
same bytes as a call of the others alone, and a time that goes with the number
of sequences."""
import pytest
import torch

from tests.rows_testlib import DTYPES, starts

pytestmark = pytest.mark.gpu

# tokens before -> new ones of the sequences that have some, and where they
# stand: blocks that the chunks go on into, taken by CTAs far from their own
MANY = [([127, 5, 127, 200, 0], [3, 1, 140, 2, 1], [0, 1, 2, 3, 4]), ([127, 127, 126, 0], [2, 2, 3, 1], [2996, 2997, 2998, 2999]),
        ([127], [2], [0]), ([127], [2], [2999]), ([100], [1], [1500]), ([1], [1100], [7]),
        ([127] * 700, [2] * 700, list(range(2300, 3000))), ([127] * 700, [2] * 700, list(range(700))),
        ([127] * 1500, [2] * 1500, list(range(0, 3000, 2)))]


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("case", range(len(MANY)))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equals_a_call_of_those_alone(case, dtype, rotary):
    import bit_quantized_kv_decode_gb300 as kvq
    old, new, at = MANY[case]
    B, wide, H, D = 3000, max((o + n + 127) // 128 for o, n in zip(old, new)), 1, 64
    desc = kvq.cache_desc(4, 1, 0, H, len(old) * wide, head_dim=D, group=32)
    g = torch.Generator(device="cuda").manual_seed(case)
    k, v = (torch.randn(sum(new), H, D, generator=g, device="cuda").to(DTYPES[dtype]) for _ in "kv")
    window = torch.randn(2, B, H, 128, D, generator=g, device="cuda")
    few_table = torch.arange(len(old) * wide, dtype=torch.int32, device="cuda").view(len(old), wide)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")  # (the others' pages are not looked at)
    table[at] = few_table
    lens, many = torch.full((B,), 77, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    lens[at], many[at] = torch.tensor(old, dtype=torch.int32), torch.tensor(new, dtype=torch.int32)
    angles = kvq.rotary_table(wide * 128, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(cu, lens, table, window, outs):
        caches = [kvq.alloc_cache(desc) for _ in "kv"]
        args = (k, v, cu.cuda(), lens.cuda(), *caches, window[0], window[1])
        kw = dict(page_table=table, k_window_out=outs[0], v_window_out=outs[1], dev_status=status)
        kvq.append_rotary(desc, angles, *args, **kw) if rotary else kvq.append_chunk(desc, *args, **kw)
        return [t.view(torch.uint8) for c in caches for t in c]

    want_outs = torch.full((2, len(old), H, 128, D), 9.0, device="cuda")
    want = call(starts(new), lens[at], few_table, window[:, at].contiguous(), want_outs)
    outs = torch.full_like(window, 9.0)
    got = call(starts(many.tolist()), lens, table, window, outs)
    assert int(status.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    idle = torch.ones(B, dtype=torch.bool, device="cuda")
    idle[at] = False
    assert torch.equal(outs[:, at], want_outs)
    assert torch.equal(outs[:, idle, :, :77], window[:, idle, :, :77]) and (outs[:, idle, :, 77:] == 9).all()


def test_time_goes_with_the_number_of_sequences():
    """A token of each of eight: four times the sequences take four times as long, not sixteen."""
    import bit_quantized_kv_decode_gb300 as kvq
    T, H, D = 8, 1, 64
    desc = kvq.cache_desc(4, 0, 0, H, T, head_dim=D, group=64)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    k, v = (torch.randn(T, H, D, device="cuda").to(torch.bfloat16) for _ in "kv")

    def time(B):
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda").clamp(max=T)
        table = torch.arange(B, dtype=torch.int32, device="cuda").clamp(max=T - 1)[:, None].contiguous()
        took = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
            a.record()
            kvq.append_chunk(desc, k, v, cu, lens, *caches, page_table=table)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        return sorted(took)[3]

    few, many = time(16383), time(65532)
    assert many <= 8 * few, f"{few * 1000:.0f} us, {many * 1000:.0f} us"

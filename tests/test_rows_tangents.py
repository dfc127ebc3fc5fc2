"""Tensors that carry a tangent (forward-mode differentiation) are refused: the
operators have no derivative, and would drop it without a word."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import bit_quantized_kv_decode_gb300 as kvq


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a GPU: the checks come first."""
    is_cuda = True


def dual(x):
    return fwd.make_dual(x, torch.ones_like(x))


@pytest.mark.parametrize("disable", [False, True])
def test_rows_with_a_tangent(disable):
    x = torch.randn(4, 2, 64).to(torch.bfloat16).as_subclass(OnDevice)
    assert kvq._rows(x, "x", kvq._HALF).data == x.data_ptr()
    with fwd.dual_level(), torch.set_grad_enabled(not disable):
        assert kvq._rows(x, "x", kvq._HALF).data == x.data_ptr()
        with pytest.raises(ValueError, match="x has a tangent"):
            kvq._rows(dual(x), "x", kvq._HALF)


@pytest.mark.gpu
def test_calls_with_a_tangent():
    T, D = 6, 128
    q, k, v = (torch.randn(T, h, D, device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    desc = kvq.cache_desc(4, 0, 0, 2, 1)
    caches = [kvq.alloc_cache(desc) for _ in "kv"]
    want = kvq.prompt_attn(q, k, v, cu)
    with fwd.dual_level():
        for call in (lambda: kvq.prompt_attn(dual(q), k, v, cu), lambda: kvq.prompt_attn(q, dual(k), v, cu),
                     lambda: kvq.prompt_attn(q, k, dual(v), cu), lambda: kvq.chunk_attn(desc, dual(q), *caches, cu, lens, max_blocks=1),
                     lambda: kvq.append_chunk(desc, dual(k), v, cu, lens, *caches, max_blocks=1),
                     lambda: kvq.append_chunk(desc, k, dual(v), cu, lens, *caches, max_blocks=1)):
            with pytest.raises(ValueError, match="tangent"):
                call()
        assert torch.equal(kvq.prompt_attn(q, k, v, cu), want)
        assert torch.equal(kvq.prompt_attn(fwd.unpack_dual(dual(q)).primal, k, v, cu), want)

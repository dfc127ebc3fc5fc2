"""The workspace of attention over lists of blocks: a call with fewer sequences or
shorter lists may take more than a larger one, so there is a size for every call."""
import pytest

import __graft_entry__ as entry
import bit_quantized_kv_decode_gb300 as kvq


@pytest.fixture(scope="module", autouse=True)
def built():
    entry.build()


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("heads,per", [(1, 1), (8, 4), (3, 2), (4, 8)])
def test_one_size_for_every_call(dim, group, heads, per):
    desc = kvq.cache_desc(4, 1, 0, heads, 64, head_dim=dim, group=group)
    most = kvq.sparse_workspace_size(desc, None, heads * per, None)
    assert most == kvq.sparse_workspace_size(desc, 7, heads * per, None) == kvq.sparse_workspace_size(desc, None, heads * per, 9)
    batches = [*range(1, 40), *(b + d for b in (64, 96, 128, 160, 256, 512, 607, 608, 1216, 2432, 4863, 9728, 65535) for d in (-1, 0)),
               65535]
    lengths = [*range(1, 40), 63, 64, 100, 128, 255, 256, 1000, 4863, 4864, 8192, 100000, 1 << 27, (1 << 30) // heads]
    sizes = {(b, n): kvq.sparse_workspace_size(desc, b, heads * per, n) for b in batches for n in lengths if b * heads * n <= 1 << 30}
    assert max(sizes.values()) <= most
    assert max(sizes.values()) >= most // 4  # (no more than what some calls take)
    assert most <= 9728 * per * (dim + 1) * 4 + 512


def test_smaller_calls_that_take_more():
    desc = kvq.cache_desc(4, 1, 0, 8, 64)
    size = {b: kvq.sparse_workspace_size(desc, b, 32, 64) for b in (96, 128, 256, 512)}
    assert size[512] < size[128] < size[96] and size[512] < size[256] <= kvq.sparse_workspace_size(desc, None, 32, None)


def test_sizes_that_are_refused():
    desc = kvq.cache_desc(3, 1, 0, 8, 64)
    for args in ((None, 32, None), (4, 32, None)):
        with pytest.raises(kvq.KvqError):
            kvq.sparse_workspace_size(desc, *args)
    with pytest.raises(kvq.KvqError):
        kvq.sparse_workspace_size(kvq.cache_desc(4, 1, 0, 8, 64), None, 24, None)

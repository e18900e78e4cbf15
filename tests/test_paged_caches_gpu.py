"""Copies in caches whose memory changes under the tensors that a list of them was made of."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("how", ["data", "set", "layout"])
def test_memory_that_changed_under_a_cache_is_where_copies_go(how):
    """The tensors are the same objects, their memory (or its layout) is another: blocks are
    copied there, and what they were before is left alone."""
    from verify_dspark_markov_step_gb300 import PagedCaches, paged_copy
    shape = (6, 2, 16, 64)
    pairs = [tuple(torch.randn(shape, device="cuda").half() for _ in range(2)) for _ in range(3)]
    caches = PagedCaches(pairs)
    copies, count = _ints([0, 1]), _ints(1)
    paged_copy(caches, copies, count)
    old = [[c.detach().view(-1) for c in pair] for pair in pairs]  # (what they were, kept alive)
    before = [[o.clone() for o in pair] for pair in old]
    changed = pairs if how == "layout" else pairs[1:]  # (the layout is one for all)
    for pair in changed:
        for c in pair:
            fresh = torch.randn(shape, device="cuda").half()
            if how == "data":
                c.data = fresh
            elif how == "set":
                c.set_(fresh)
            else:  # the same memory, the blocks interleaved
                c.as_strided_(shape, (64, 6 * 16 * 64, 6 * 64, 1))
    want = [[c.clone() for c in pair] for pair in pairs]
    for pair in want:
        for c in pair:
            c[3] = c[2]
    paged_copy(caches, _ints([2, 3]), count)
    torch.cuda.synchronize()
    for pair, expect in zip(pairs, want):
        assert all(torch.equal(a, b) for a, b in zip(pair, expect))
    if how != "layout":
        for was, now in zip(before[1:], old[1:]):
            assert all(torch.equal(a, b) for a, b in zip(was, now))


def test_a_paged_cache_follows_its_memory():
    from verify_dspark_markov_step_gb300.paged import PagedCache
    cache = PagedCache(layers=2, slots=3, max_len=64, num_blocks=12, page_size=16, q_heads=2, kv_heads=2, head_dim=64)
    cache.plan(_ints(0), _ints(20), 20)
    cache.cached_lens[0] = 20
    cache.fork(_ints(0), _ints(1))
    old = [c.detach() for c in cache.k + cache.v]
    kept = [c.view(c.shape) for c in old]
    before = [c.clone() for c in kept]
    for c in cache.k + cache.v:
        c.data = torch.randn_like(c)
    cache.fork(_ints(0), _ints(2))
    torch.cuda.synchronize()
    a, b = cache.block_table[0, :2].long(), cache.block_table[2, :2].long()
    assert cache.status_code() == 0
    for c in cache.k + cache.v:
        assert torch.equal(c[a], c[b])
    assert all(torch.equal(x, y) for x, y in zip(kept, before))

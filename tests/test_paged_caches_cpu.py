"""A list of caches for the copies, without a GPU: tensors that say they are on one."""
import pytest
import torch

from verify_dspark_markov_step_gb300 import _lib


class There(torch.Tensor):
    """A host tensor that answers as one on a GPU."""
    device_index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.device_index


class Elsewhere(There):
    device_index = 1


def _cache(kind=There, blocks=4):
    return torch.zeros(blocks, 2, 16, 64, dtype=torch.float16).as_subclass(kind)


def _addresses(caches):
    return [(kv.k, kv.v) for kv in caches.array]


def test_a_list_notices_what_changes_under_its_tensors():
    pairs = [(_cache(), _cache()) for _ in range(3)]
    caches = _lib.PagedCaches(pairs)
    before, array = _addresses(caches), caches.array
    caches.look()
    assert caches.array is array  # nothing has changed
    kept, fresh = pairs[1][0].data, _cache()
    pairs[1][0].data = fresh
    caches.look()
    assert _addresses(caches)[1] == (fresh.data_ptr(), before[1][1]) and kept.data_ptr() == before[1][0]
    assert [_addresses(caches)[i] for i in (0, 2)] == [before[i] for i in (0, 2)]
    fresh = _cache(blocks=9)
    for c in pairs[2]:
        c.data = fresh
    caches.look()
    assert caches.array[2].num_blocks == 9
    strides = (64, 4 * 16 * 64, 4 * 64, 1)
    pairs[0][0].as_strided_(pairs[0][0].shape, strides)
    caches.look()
    got = caches.array[0]
    assert (got.k_block_stride, got.k_head_stride, got.k_token_stride) == strides[:3]


def test_caches_of_two_devices_are_refused():
    with pytest.raises(ValueError, match="one device"):
        _lib.PagedCaches([(_cache(), _cache()), (_cache(), _cache(Elsewhere))])
    with pytest.raises(ValueError, match="one device"):
        _lib.PagedCaches([(_cache(), _cache()), (_cache(Elsewhere), _cache(Elsewhere))])


def test_copies_on_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_lib", object())  # (no call is made)
    caches = [(_cache(), _cache())]
    copies = torch.zeros(3, 2, dtype=torch.int32).as_subclass(Elsewhere)
    count = torch.zeros(1, dtype=torch.int32).as_subclass(Elsewhere)
    for c in (caches, _lib.PagedCaches(caches)):
        with pytest.raises(ValueError, match="device"):
            _lib.paged_copy(c, copies, count)
    with pytest.raises(TypeError, match="CUDA"):
        _lib.paged_copy(caches, torch.zeros(3, 2, dtype=torch.int32), count)


def test_a_paged_cache_keeps_no_replaced_tensor(monkeypatch):
    """Caches that are replaced, added or given up are the ones copied, and their memory goes."""
    import types
    import weakref

    from verify_dspark_markov_step_gb300.paged import PagedCache
    cache = PagedCache(layers=2, slots=3, max_len=64, num_blocks=4, page_size=16, q_heads=2, kv_heads=2, head_dim=64,
                       dtype=torch.float16, device="cpu")
    cache.k, cache.v = ([_cache() for _ in range(2)] for _ in range(2))
    cache.copies, cache.copied = (t.as_subclass(There) for t in (cache.copies, cache.copied))
    cache.status = cache.status.as_subclass(There)
    seen = []

    def copy(array, n, *a):
        seen.append([(kv.k, kv.v) for kv in array[:n]])
        return 0
    monkeypatch.setattr(_lib, "_lib", types.SimpleNamespace(dspark_paged_copy=copy))
    monkeypatch.setattr(_lib, "_stream_here", lambda *a: 0)
    monkeypatch.setattr(_lib, "paged_fork", lambda *a, **kw: None)

    def now():
        return [(k.data_ptr(), v.data_ptr()) for k, v in zip(cache.k, cache.v)]
    slots = torch.zeros(1, dtype=torch.int32)
    cache.fork(slots, slots)
    assert seen[-1] == now()
    gone = weakref.ref(cache.k[1])
    cache.k[1] = _cache()
    assert gone() is None
    cache.k.append(_cache()), cache.v.append(_cache())
    cache.fork(slots, slots)
    assert seen[-1] == now() and len(seen[-1]) == 3
    gone = [weakref.ref(t) for t in cache.k]
    cache.k, cache.v = [], []
    assert not any(g() is not None for g in gone)

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

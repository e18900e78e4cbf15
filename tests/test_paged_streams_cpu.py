"""Which stream the paged cache's own work and memory belong to, without a GPU: the
library calls and torch's current stream are recorded, nothing is computed on a
device."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
from torch.overrides import TorchFunctionMode  # noqa: E402


class Side:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def rec(monkeypatch):
    """.calls: (library call, stream argument, workspace); .ops: the current stream of
    every torch operation; .made: the current stream of every workspace."""
    from verify_dspark_markov_step_gb300 import _lib

    r = types.SimpleNamespace(calls=[], ops=[], made=[], now=[None])

    @contextlib.contextmanager
    def stream(s):
        r.now.append(r.now[-1] if s is None else s)
        yield
        r.now.pop()

    def call(name):
        def f(*a, stream=None, workspace_buf=None, **kw):
            r.calls.append((name, r.now[-1] if stream is None else stream, workspace_buf))
        return f

    def workspace(n, device="cuda"):
        r.made.append(r.now[-1])
        return torch.empty(8)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("paged_tables", "kv_append", "paged_attention"):
        monkeypatch.setattr(_lib, name, call(name))
    monkeypatch.setattr(_lib, "workspace", workspace)
    monkeypatch.setattr(_lib, "paged_attention_workspace_bytes", lambda *a: 8)
    monkeypatch.setattr(_lib, "_raw_stream", lambda s, t: (
        s or r.now[-1] or Side(0)).cuda_stream)
    return r


def _cache(layers=2):
    from verify_dspark_markov_step_gb300.paged import PagedCache
    return PagedCache(layers=layers, slots=3, max_len=64, num_blocks=8, page_size=16, q_heads=4,
                      kv_heads=2, head_dim=64, device="cpu")


class Ops(TorchFunctionMode):
    def __init__(self, r):
        super().__init__()
        self.r = r

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.r.ops.append((getattr(func, "__name__", str(func)), self.r.now[-1]))
        return func(*args, **(kwargs or {}))


def test_the_targets_forward_runs_on_one_stream(rec):
    from verify_dspark_markov_step_gb300.paged import ToyTarget
    target = ToyTarget(32, 2, 4, 2, 64, dtype=torch.float32, device="cpu")
    cache, side = _cache(), Side(5)
    rsi = torch.zeros(1, dtype=torch.int32)
    cache.plan(rsi, rsi + 3, 3, stream=side)
    with Ops(rec):
        target.forward(torch.tensor([1, 2, 3]), cache, stream=side)
    names = {n for n, _ in rec.ops}
    assert "matmul" in names or "__matmul__" in names, names
    work = [(n, s) for n, s in rec.ops if n not in ("tensor", "__get__", "device")]
    assert len(work) > 10 and all(s is side for _, s in work)
    assert len(rec.calls) == 5 and all(s is side for _, s, _ in rec.calls)
    rec.ops.clear(), rec.calls.clear()
    with Ops(rec):
        target.forward(torch.tensor([1, 2, 3]), cache)
    assert all(s is None for _, s in rec.ops) and all(s is None for _, s, _ in rec.calls)


def test_a_workspace_belongs_to_the_stream_that_uses_it(rec):
    cache = _cache()
    rsi = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64)
    one, two = Side(5), Side(6)
    cache.plan(rsi, rsi + 1, 1)
    for s in (None, one, two, one, None):
        cache.attend(0, q, q.clone(), stream=s)
    with torch.cuda.stream(two):
        cache.attend(1, q, q.clone())
    used = [w for n, _, w in rec.calls if n == "paged_attention"]
    assert used[0] is used[4] and used[1] is used[3] and used[2] is used[5]
    assert len({id(w) for w in used}) == 3
    assert rec.made == [None, one, two]


def test_plans_of_many_sizes_share_their_buffers(rec):
    """Lengths of prompts vary without end: the plans' buffers stay within four times
    the largest plan, and none is freed (a captured graph may still write to it)."""
    cache = _cache()
    rsi = torch.zeros(3, dtype=torch.int32)
    kept, storages = [], {}
    for T in [4096, 1, 7, *range(1000, 4000, 7), 0, 4096]:
        for B in (1, 2, 3):
            made = cache.plan(rsi[:B], rsi[:B], T)
            assert [tuple(t.shape) for t in made] == [(B + 1,), (B,), (T,), (T,)]
            assert [t.dtype for t in made] == [torch.int32] * 2 + [torch.int64] * 2
            assert all(t.is_contiguous() for t in made) and made is cache.step
            for t in made:
                storages[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
            kept.append(made)
    assert sum(storages.values()) <= 4 * (2 * 8 * 4096) + 2 * 4 * 1025
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(kept[2], kept[-1]))

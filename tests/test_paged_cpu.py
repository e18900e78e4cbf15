"""The paged-cache calls without a GPU: host-side refusals of the C ABI and of
the binding, and the tables' statement against properties it has to have."""
import ctypes
import os
import random
import shutil

import pytest

import paged_oracle as po


@pytest.fixture(scope="module")
def L():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from verify_dspark_markov_step_gb300 import build, _lib
    build.build()
    return _lib.lib()


FAKE = ctypes.c_void_p(4096)  # never dereferenced: every call below fails on the host


def _cache(**kw):
    from verify_dspark_markov_step_gb300 import _lib
    d = dict(k=4096, v=4096, k_scale=None, v_scale=None, k_block_stride=8 * 16 * 128,
             k_head_stride=16 * 128, k_token_stride=128, v_block_stride=8 * 16 * 128,
             v_head_stride=16 * 128, v_token_stride=128, dtype=1, num_blocks=10, kv_heads=8,
             page_size=16, head_dim=128)
    d.update(kw)
    return _lib.PagedKv(**d)


def test_tables_refusals(L):
    def call(B=1, S=1, M=4, N=8, T=16, page=16, table=FAKE, start=FAKE, slot=FAKE):
        return L.dspark_paged_tables(FAKE, FAKE, FAKE, None, table, FAKE, FAKE, FAKE, start, FAKE,
                                     FAKE, slot, B, S, M, N, T, page, None, None)
    assert call(B=-1) == -1
    assert call(B=1025) == -1
    assert call(S=0) == -1
    assert call(M=0) == -1
    assert call(M=(1 << 20) + 1) == -1
    assert call(N=0) == -1
    assert call(T=-1) == -1
    assert call(page=8) == -2
    assert call(page=48) == -2
    assert call(page=512) == -2
    assert call(table=None) == -1
    assert call(start=None) == -1
    assert call(slot=None) == -1


def test_append_refusals(L):
    def call(T=4, dtype=1, ks=1024, k=FAKE, slot=FAKE, cache=None, **kw):
        c = _cache(**kw) if cache is None else cache
        return L.dspark_kv_append(k, FAKE, dtype, ks, 1024, c, slot, T, None, None)
    assert call(T=-1) == -1
    assert L.dspark_kv_append(FAKE, FAKE, 1, 1024, 1024, None, FAKE, 4, None, None) == -1
    assert call(k=None) == -1
    assert call(slot=None) == -1
    assert call(dtype=0) == -1
    assert call(dtype=3) == -1
    assert call(dtype=2) == -2            # fp16 rows, bf16 cache
    assert call(num_blocks=0) == -1
    assert call(kv_heads=0) == -1
    assert call(page_size=24) == -2
    assert call(head_dim=96) == -2
    assert call(k=ctypes.c_void_p(4098)) == -7
    assert call(ks=1028) == -7
    assert call(v_token_stride=132) == -7
    assert call(dtype=1, k_head_stride=-16) == -7
    assert call(v=4100) == -7
    # an 8-bit cache counts its strides in bytes
    assert call(cache=_cache(dtype=3, k_token_stride=136)) == -7
    assert call(T=0) == 0


def test_attention_refusals(L):
    ws = L.dspark_paged_attention_workspace_bytes(1, 32, 8, 128)
    assert ws > 0
    assert L.dspark_paged_attention_workspace_bytes(-1, 32, 8, 128) == 0
    assert L.dspark_paged_attention_workspace_bytes(1, 33, 8, 128) == 0
    assert L.dspark_paged_attention_workspace_bytes(1, 32, 8, 80) == 0

    def call(B=1, S=1, M=4, T=4, Hq=32, dtype=1, qs=4096, scale=0.1, causal=1, window=0, q=FAKE,
             out=FAKE, w=FAKE, wb=ws, **kw):
        return L.dspark_paged_attention(q, dtype, qs, _cache(**kw), FAKE, FAKE, FAKE, FAKE, out,
                                        None, scale, causal, window, Hq, B, S, M, T, w, wb, None,
                                        None)
    assert call(B=-1) == -1
    assert call(B=1025) == -1
    assert call(S=0) == -1
    assert call(M=0) == -1
    assert call(T=-1) == -1
    assert call(T=1 << 24) == -1
    assert call(Hq=0) == -1
    assert call(Hq=33) == -1
    assert call(Hq=8 * 129) == -2
    assert call(dtype=0) == -1
    assert call(dtype=2) == -2
    assert call(scale=float("nan")) == -1
    assert call(scale=float("inf")) == -1
    assert call(causal=2) == -1
    assert call(window=-1) == -1
    assert call(head_dim=256) == -2
    assert call(page_size=512) == -2
    assert call(q=None) == -1
    assert call(out=None) == -1
    assert call(q=ctypes.c_void_p(4104)) == -7
    assert call(qs=4100) == -7
    assert call(w=None) == -6
    assert call(wb=ws - 1) == -6
    assert call(B=0) == 0
    assert call(T=0) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    from verify_dspark_markov_step_gb300 import _lib
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        _lib.kv_append(q, q, c, c, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError, match="CUDA"):
        _lib.paged_attention(q, c, c, i[None], i, i, i, q)
    with pytest.raises(TypeError, match="CUDA"):
        _lib.paged_tables(i, i, i, i[None], i, i, i, i, i, i, i, 16)


def test_tables_statement_keeps_the_blocks():
    """Over random steps no block is lost or held twice, every live position
    has its own slot, and a step taken back leaves the stack as it was."""
    r = random.Random(5)
    page, S, M, N = 16, 7, 9, 40
    table, held, cached = [[-1] * M for _ in range(S)], [0] * S, [0] * S
    free, count = list(range(N)), N
    r.shuffle(free)
    for step in range(200):
        rsi = r.sample(range(S), 5)
        rsi[r.randrange(5)] = -1
        new = [r.choice((0, 1, 3, 17, 40)) for _ in rsi]
        if step % 4 == 3:  # requests that ended
            for s in r.sample(range(S), 2):
                cached[s] = 0
        o = po.tables(rsi, new, cached, None, table, held, free, count, 120, page)
        owned = [o["block_table"][s][j] for s in range(S) for j in range(o["held_blocks"][s])]
        assert sorted(owned + o["stack"]) == list(range(N))
        live = [x for x in o["slot_map"] if x >= 0]
        assert len(live) == len(set(live))
        back = po.tables(rsi, [0] * 5, cached, None, o["block_table"], o["held_blocks"],
                         o["stack"], len(o["stack"]), 120, page)
        if all(h <= -(-cached[s] // page) for s, h in enumerate(held)):
            again = po.tables(rsi, [0] * 5, cached, None, table, held, free, count, 120, page)
            assert back["stack"] == again["stack"]
        table, held = o["block_table"], o["held_blocks"]
        free, count = o["stack"] + [0] * (N - len(o["stack"])), len(o["stack"])
        for b, s in enumerate(rsi):
            if s >= 0 and o["seq_lens"][b]:
                cached[s] = r.randint(cached[s], o["seq_lens"][b])

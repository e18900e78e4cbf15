"""Forking, freeing, compacting and copying without a GPU: refusals of the C ABI, and
the plain statement against what always has to hold."""
import ctypes
import os
import random
import shutil

import pytest

import paged_blocks_oracle as bo


@pytest.fixture(scope="module")
def L():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from verify_dspark_markov_step_gb300 import build, _lib
    build.build()
    return _lib.lib()


FAKE = ctypes.c_void_p(4096)  # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p(4100)


def test_fork_refusals(L):
    def call(src=FAKE, dst=FAKE, lens=FAKE, table=FAKE, held=FAKE, free=FAKE, pool=FAKE, shares=None,
             copies=FAKE, count=FAKE, n=1, S=4, M=4, N=8, C=8, page=16):
        return L.dspark_paged_fork(src, dst, lens, table, held, free, pool, shares, copies, count, n,
                                   S, M, N, C, page, None, None)
    for kw in ({"n": -1}, {"n": 1025}, {"S": 0}, {"M": 0}, {"M": (1 << 20) + 1}, {"N": 0},
               {"N": 1 << 30}, {"C": -1}, {"C": 1 << 30}):
        assert call(**kw) == -1, kw
    for name in ("src", "dst", "lens", "table", "held", "free", "pool", "copies", "count"):
        assert call(**{name: None}) == -1, name
    assert call(page=8) == -2
    assert call(page=48) == -2
    assert call(copies=ODD) == -7


def test_free_refusals(L):
    def call(slots=FAKE, lens=FAKE, table=FAKE, held=FAKE, free=FAKE, pool=FAKE, n=1, S=4, M=4, N=8):
        return L.dspark_paged_free(slots, lens, table, held, free, pool, None, n, S, M, N, None, None)
    for kw in ({"n": -1}, {"n": 1025}, {"S": 0}, {"M": 0}, {"N": 0}):
        assert call(**kw) == -1, kw
    for name in ("slots", "lens", "table", "held", "free", "pool"):
        assert call(**{name: None}) == -1, name
    assert call(n=0, slots=None) == 0


def test_compact_refusals(L):
    assert L.dspark_paged_compact_workspace_bytes(0) == 0
    assert L.dspark_paged_compact_workspace_bytes(1000) >= 4000

    def call(table=FAKE, held=FAKE, free=FAKE, pool=FAKE, copies=FAKE, count=FAKE, S=4, M=4, N=8, C=4,
             ws=FAKE, size=4096):
        return L.dspark_paged_compact(table, held, free, pool, None, copies, count, S, M, N, C, ws,
                                      size, None, None)
    for kw in ({"S": 0}, {"M": 0}, {"N": 0}, {"C": 3}, {"N": 9, "C": 3}):
        assert call(**kw) == -1, kw
    for name in ("table", "held", "free", "pool", "copies", "count"):
        assert call(**{name: None}) == -1, name
    assert call(copies=ODD) == -7
    assert call(ws=None) == -6
    assert call(size=16) == -6
    assert call(ws=ctypes.c_void_p(4104)) == -6


def test_copy_refusals(L):
    from verify_dspark_markov_step_gb300 import _lib

    def cache(**kw):
        d = dict(k=4096, v=4096, k_scale=None, v_scale=None, k_block_stride=8 * 16 * 128,
                 k_head_stride=16 * 128, k_token_stride=128, v_block_stride=8 * 16 * 128,
                 v_head_stride=16 * 128, v_token_stride=128, dtype=1, num_blocks=10, kv_heads=8,
                 page_size=16, head_dim=128)
        d.update(kw)
        return _lib.PagedKv(**d)

    def call(*caches, n=None, copies=FAKE, count=FAKE, C=4):
        a = (_lib.PagedKv * max(1, len(caches)))(*caches)
        return L.dspark_paged_copy(a, len(caches) if n is None else n, copies, count, C, None, None)
    assert call(cache(), n=-1) == -1
    assert L.dspark_paged_copy(None, 1, FAKE, FAKE, 4, None, None) == -1
    assert call(cache(), C=-1) == -1
    assert call(cache(), copies=None) == -1
    assert call(cache(), count=None) == -1
    assert call(cache(), copies=ODD) == -7
    assert call(cache(k=None)) == -1
    assert call(cache(), cache(v=4100)) == -7
    assert call(cache(page_size=24)) == -2
    for kw in ({"num_blocks": 9}, {"kv_heads": 4}, {"page_size": 32}, {"head_dim": 64}, {"dtype": 2},
               {"k_block_stride": 8 * 16 * 256}, {"v_token_stride": 256}, {"k_head_stride": 64}):
        assert call(cache(), cache(**kw)) == -2, kw
    assert call() == 0
    assert call(cache(), C=0) == 0


def test_shared_tables_refusals(L):
    def call(table=FAKE, shares=FAKE, B=1, page=16):
        return L.dspark_paged_tables_shared(FAKE, FAKE, FAKE, None, table, FAKE, FAKE, FAKE, shares,
                                            FAKE, FAKE, FAKE, FAKE, B, 4, 4, 8, 16, page, None, None)
    assert call(B=1025) == -1
    assert call(table=None) == -1
    assert call(page=24) == -2


@pytest.mark.parametrize("sharing", [False, True])
def test_plain_statement_keeps_its_invariants(sharing):
    for seed in range(60):
        rng = random.Random(seed)
        S, M, N, page = rng.randint(2, 9), rng.randint(1, 6), rng.randint(4, 40), rng.choice((16, 32))
        stack = list(range(N))
        rng.shuffle(stack)
        t = {"table": [[-1] * M for _ in range(S)], "held": [0] * S, "cached": [0] * S, "stack": stack,
             "shares": [0] * N if sharing else None, "N": N}
        for s in range(S // 2):
            n = rng.randint(0, min(M, len(stack)) * page)
            for j in range(-(-n // page)):
                t["table"][s][j] = t["stack"].pop()
            t["held"][s], t["cached"][s] = -(-n // page), n
        bo.check(t)
        for _ in range(12):
            k = rng.randint(0, 4)
            if rng.random() < 0.5:
                before = [list(t["stack"]), [list(r) for r in t["table"]]]
                src, dst = ([rng.randint(-1, S) for _ in range(k)] for _ in range(2))
                copies, codes = bo.fork(t, src, dst, page, rng.choice((2, 100)))
                assert len({b for _, b in copies}) == len(copies)
                assert not {a for a, _ in copies} & {b for _, b in copies}
                made = [d for s, d in zip(src, dst) if s >= 0 and d >= 0]
                if not codes and rng.random() < 0.5:  # taken back whole
                    bo.check(t)
                    assert not bo.free(t, made)
                    assert [t["stack"], t["table"]] == before
            elif rng.random() < 0.6:
                bo.free(t, [rng.randint(-1, S) for _ in range(k)])
            else:
                moves = bo.compact(t)
                assert all(a > b for a, b in moves)
                used = N - len(t["stack"])
                assert all(b < used for r, n in zip(t["table"], t["held"]) for b in r[:n])
            bo.check(t)

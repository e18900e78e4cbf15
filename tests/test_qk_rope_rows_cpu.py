"""Where the rotating calls write rows, without a GPU: rows that overlap each other, or rows
that are read, are refused."""
import os
import shutil

import pytest

from verify_dspark_markov_step_gb300 import _lib

BASE = 1 << 20  # addresses that are never dereferenced


@pytest.fixture(scope="module")
def L():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from verify_dspark_markov_step_gb300 import build
    build.build()
    return _lib.lib()


# (where the rows go, in bytes from those that are read; stride read, stride written; T) with
# rows of 8 heads of 128: 1024 values, 2048 bytes. Strides in values.
REFUSED = [(0, 1024, 2048, 4), (0, 2048, 1024, 4), (0, 512, 512, 2), (1 << 30, 1024, 1016, 4), (1 << 30, 1024, 8, 2),
           (16, 1024, 1024, 4), (-16, 1024, 1024, 4), (2048, 1024, 1024, 4), (-2048, 1024, 1024, 2), (256, 2048, 2048, 3),
           (2032, 2048, 2048, 3), (2064, 2048, 2048, 3), (4096 - 2032, 2048, 2048, 3), (16, 1024, 1024, 1),
           (-2032, 4096, 512, 1), (4096, 1024, 2048, 4), (2048, 4096, 1024, 4), (4096 * 2 + 16, 2048, 2048, 3)]


def _rows_call(L, off, qs, qos, T, keys):
    q, k = (1 << 40, BASE) if keys else (BASE, 1 << 40)
    out = BASE + (1 << 35) + off if abs(off) >= 1 << 30 else BASE + off
    other = (1 << 41, 1024, 1024)
    mine = (out, qs, qos)
    (qo, q1, q2), (ko, k1, k2) = (other, mine) if keys else (mine, other)
    return L.dspark_qk_rope(q, qo, k, ko, 1, q1, q2, k1, k2, BASE, BASE, 1.0, 64, 0, None, None, 1e-6, 8, 8, 128, T, None)


@pytest.mark.parametrize("keys", [False, True])
@pytest.mark.parametrize("off,qs,qos,T", REFUSED)
def test_rows_that_overlap_are_refused(L, off, qs, qos, T, keys):
    assert _rows_call(L, off, qs, qos, T, keys) == -1


@pytest.mark.parametrize("off,qs,qos,T", REFUSED)
def test_queries_beside_the_pages_too(L, off, qs, qos, T):
    c = _lib.PagedKv(k=BASE, v=BASE, k_scale=None, v_scale=None, k_block_stride=8 * 16 * 128, k_head_stride=16 * 128,
                     k_token_stride=128, v_block_stride=8 * 16 * 128, v_head_stride=16 * 128, v_token_stride=128, dtype=1,
                     num_blocks=10, kv_heads=8, page_size=16, head_dim=128)
    out = BASE + (1 << 35) + off if abs(off) >= 1 << 30 else BASE + off
    assert L.dspark_qk_rope_append(BASE, out, 1 << 40, 1 << 40, 1, qs, qos, 1024, 1024, c, BASE, BASE, BASE, 1.0, 64, 0, None,
                                   None, 1e-6, 8, T, None, None) == -1

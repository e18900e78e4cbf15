"""Refusals of the attention with sinks, and its visible keys by hand."""
import ctypes
import os
import shutil

import pytest

import paged_sinks_oracle as so


def test_refusals():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from verify_dspark_markov_step_gb300 import build, _lib
    build.build()
    L = _lib.lib()
    fake = ctypes.c_void_p(4096)  # never dereferenced: every call below fails on the host
    c = _lib.PagedKv(k=4096, v=4096, k_scale=None, v_scale=None, k_block_stride=8 * 16 * 128,
                     k_head_stride=16 * 128, k_token_stride=128, v_block_stride=8 * 16 * 128,
                     v_head_stride=16 * 128, v_token_stride=128, dtype=1, num_blocks=10, kv_heads=8,
                     page_size=16, head_dim=128)

    def call(window=100, sinks=4, ws=1 << 30, B=1, q=fake, scale=0.1):
        return L.dspark_paged_attention_sinks(q, 1, 4096, c, fake, fake, fake, fake, fake, None, scale, 1,
                                              window, sinks, 32, B, 1, 4, 8, fake, ws, None, None)
    assert call(sinks=-1) == -1
    assert call(window=-1) == -1
    assert call(scale=float("nan")) == -1
    assert call(q=None) == -1
    assert call(ws=1024) == -6
    assert call(B=0) == 0


def test_visible_keys():
    import torch
    got = so.visible(3, 8, True, 2, 2, "cpu").int().tolist()
    assert got == [[1, 1, 0, 0, 1, 1, 0, 0], [1, 1, 0, 0, 0, 1, 1, 0], [1, 1, 0, 0, 0, 0, 1, 1]]
    got = so.visible(2, 5, False, 2, 1, "cpu").int().tolist()
    assert got == [[1, 0, 1, 1, 1], [1, 0, 0, 1, 1]]
    assert so.visible(2, 5, True, 0, 1, "cpu").int().tolist() == [[1, 1, 1, 1, 0], [1] * 5]
    assert torch.equal(so.visible(3, 2, True, 5, 1, "cpu").int(), torch.tensor([[0, 0], [1, 0], [1, 1]]))

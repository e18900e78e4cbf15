"""Workspaces in host memory are refused before a call, without a GPU."""
import types

import pytest
import torch

from test_paged_caches_cpu import There
from verify_dspark_markov_step_gb300 import _lib


def _there(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(There)


@pytest.fixture
def calls(monkeypatch):
    made = []

    def call(name, result=0):
        return lambda *a: made.append(name) or result
    fake = types.SimpleNamespace(dspark_paged_compact=call("compact"), dspark_paged_attention_sinks=call("attention"),
                                 dspark_rejection_sample=call("verify"),
                                 dspark_verify_workspace_bytes=call("size", 64))
    monkeypatch.setattr(_lib, "_lib", fake)
    monkeypatch.setattr(_lib, "lib", lambda: fake)
    monkeypatch.setattr(_lib, "_stream_here", lambda *a: 0)
    monkeypatch.setattr(_lib, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(_lib, "_stream", lambda *a: 0)
    return made


def _compact(ws):
    _lib.paged_compact(_there(2, 3), _there(2), _there(8), _there(2), _there(8, 2), _there(1), workspace_buf=ws)


def _attend(ws):
    f16 = torch.float16
    q, cache = _there(4, 2, 64, dtype=f16), _there(3, 2, 16, 64, dtype=f16)
    _lib.paged_attention(q, cache, cache, _there(1, 3), _there(1), _there(2), _there(1), _there(4, 2, 64, dtype=f16),
                         workspace_buf=ws)


def _verify(ws):
    f32, i64 = torch.float32, torch.int64
    _lib.rejection_sample(_there(1, 2), None, _there(1, 3, 8, dtype=f32), _there(1), _there(1, dtype=i64), _there(1, dtype=f32),
                          _there(1, dtype=f32), _there(1, dtype=torch.uint64), _there(1, 3), _there(1), workspace_buf=ws)


@pytest.mark.parametrize("call", [_compact, _attend, _verify])
def test_a_workspace_is_the_gpus(call, calls):
    with pytest.raises(TypeError, match="workspace"):
        call(torch.zeros(4096, dtype=torch.uint8))
    assert not set(calls) - {"size"}
    call(_there(4096, dtype=torch.uint8))
    assert set(calls) - {"size"}

"""Thin ctypes binding of the C ABI in ``include/dspark.h``.

Argument marshalling only: every step of the computation runs in the CUDA
library ``_build/libdspark.so``. PyTorch provides device memory and the
current stream. There is no CPU fallback: if the library cannot be loaded,
every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libdspark.so")

DSPARK_F32 = 0
DSPARK_BF16 = 1
DSPARK_F16 = 2
DSPARK_E4M3 = 3

STATUS = {
    0: "DSPARK_OK",
    -1: "DSPARK_ERR_INVALID_ARG",
    -2: "DSPARK_ERR_UNSUPPORTED",
    -3: "DSPARK_ERR_CUDA",
    -4: "DSPARK_ERR_TIMEOUT",
    -5: "DSPARK_ERR_BOUNDS",
    -6: "DSPARK_ERR_WORKSPACE",
    -7: "DSPARK_ERR_ALIGNMENT",
    -8: "DSPARK_ERR_SCRATCH_LIMIT",
    -9: "DSPARK_ERR_CACHE_FULL",
}

# Every symbol include/dspark.h and include/dspark_testing.h declare.
EXPORTS = (
    "dspark_testing_markov_wait_limit",
    "dspark_testing_temperature_divide",
    "dspark_markov_workspace_bytes",
    "dspark_markov_sample",
    "dspark_markov_sample_static",
    "dspark_markov_topk_workspace_bytes",
    "dspark_markov_sample_topk",
    "dspark_verify_workspace_bytes",
    "dspark_rejection_sample",
    "dspark_noise",
    "dspark_paged_tables",
    "dspark_kv_append",
    "dspark_paged_attention_workspace_bytes",
    "dspark_paged_attention",
    "dspark_status_string",
    "dspark_version",
)


class PagedKv(ctypes.Structure):
    """dspark_paged_kv (see include/dspark.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [(f"{c}_{n}_stride", ctypes.c_int64) for c in "kv"
                   for n in ("block", "head", "token")]
                + [(n, ctypes.c_int32) for n in ("dtype", "num_blocks", "kv_heads", "page_size",
                                                 "head_dim")])


class DsparkError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


_lock = threading.Lock()
_lib = None


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load libdspark.so (built by ``verify_dspark_markov_step_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library not built: {p} is missing. Run "
                "`python -m verify_dspark_markov_step_gb300.build` (needs nvcc).")
        L = ctypes.CDLL(p)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.dspark_markov_workspace_bytes.restype = sz
        L.dspark_markov_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.dspark_markov_sample.restype = i32
        L.dspark_markov_sample.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp,
                                           vp, i32, i32, i32, i32, i32, i32, vp, sz, vp, vp]
        L.dspark_testing_markov_wait_limit.restype = i32
        L.dspark_testing_markov_wait_limit.argtypes = [
            vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
            vp, sz, vp, vp, ctypes.c_uint64, ctypes.c_uint32]
        L.dspark_testing_temperature_divide.restype = i32
        L.dspark_testing_temperature_divide.argtypes = [vp, vp, vp, i64, vp]
        L.dspark_markov_sample_static.restype = i32
        L.dspark_markov_sample_static.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                                  vp, vp, vp, i32, i32, i32, i32, i32, i32, vp,
                                                  vp]
        L.dspark_markov_topk_workspace_bytes.restype = sz
        L.dspark_markov_topk_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.dspark_markov_sample_topk.restype = i32
        L.dspark_markov_sample_topk.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp,
                                                vp, i32, i32, i32, i32, i32, i32, i32, vp, sz,
                                                vp, vp]
        L.dspark_verify_workspace_bytes.restype = sz
        L.dspark_verify_workspace_bytes.argtypes = [i32, i32, i32]
        L.dspark_rejection_sample.restype = i32
        L.dspark_rejection_sample.argtypes = [vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp,
                                              vp, vp, i32, i32, i32, i32, i32, vp, sz, vp, vp]
        L.dspark_noise.restype = i32
        L.dspark_noise.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, vp]
        kvp = ctypes.POINTER(PagedKv)
        L.dspark_paged_tables.restype = i32
        L.dspark_paged_tables.argtypes = [vp] * 12 + [i32] * 6 + [vp, vp]
        L.dspark_kv_append.restype = i32
        L.dspark_kv_append.argtypes = [vp, vp, i32, i64, i64, kvp, vp, i32, vp, vp]
        L.dspark_paged_attention_workspace_bytes.restype = sz
        L.dspark_paged_attention_workspace_bytes.argtypes = [i32] * 4
        L.dspark_paged_attention.restype = i32
        L.dspark_paged_attention.argtypes = [vp, i32, i64, kvp, vp, vp, vp, vp, vp, vp,
                                             ctypes.c_float, i32, i32, i32, i32, i32, i32, i32,
                                             vp, sz, vp, vp]
        L.dspark_status_string.restype = ctypes.c_char_p
        L.dspark_status_string.argtypes = [i32]
        L.dspark_version.restype = i32
        L.dspark_version.argtypes = []
        if path is None:
            _lib = L
        return L


def status_string(code: int) -> str:
    return lib().dspark_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, dtypes=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    return t


_BF16_LIKE = (torch.bfloat16, torch.int16)


def _logit_dtype(t, name):
    if t.dtype == torch.float32:
        return DSPARK_F32
    if t.dtype in _BF16_LIKE:
        return DSPARK_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _check(code, what):
    if code != 0:
        raise DsparkError(code, what)


def markov_workspace_bytes(B, K, V, R) -> int:
    return int(lib().dspark_markov_workspace_bytes(B, K, V, R))


def verify_workspace_bytes(B, K, V) -> int:
    return int(lib().dspark_verify_workspace_bytes(B, K, V))


ROW_STATS_BYTES = 16  # sizeof(dspark_row_stats)


def row_stats(B: int, K: int, device=None) -> torch.Tensor:
    """A device buffer for [B, K] dspark_row_stats (16 bytes each: the row
    maximum as fp32 in the low word, a scratch word, the fixed-point mass)."""
    return torch.zeros((B, K, 2), dtype=torch.int64, device=device or "cuda")


def row_stats_fields(t: torch.Tensor):
    """(m [B,K] fp32, mass [B,K] int64) of a row_stats buffer, on the host."""
    a = t.cpu()
    m = a[..., 0].to(torch.int64).bitwise_and(0xFFFFFFFF).to(torch.int32).view(torch.float32)
    return m, a[..., 1]


def _stats(t, B, K, name="draft_stats"):
    if t is None:
        return None
    _dev(t, name)
    if t.numel() * t.element_size() != B * K * ROW_STATS_BYTES:
        raise ValueError(f"{name} must hold [B, K] {ROW_STATS_BYTES}-byte records")
    return t


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A device byte buffer usable as a workspace."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device or "cuda")


def markov_sample(base_logits, markov_w1, markov_w2, anchor_tokens, req_state_idx,
                  positions, temperature, seeds, out_tokens, cache=None,
                  cache_row_map=None, workspace_buf=None, status=None, stream=None,
                  draft_stats=None):
    """dspark_markov_sample on torch tensors (see include/dspark.h)."""
    _dev(base_logits, "base_logits", (torch.float32,) + _BF16_LIKE)
    B, K, V = base_logits.shape
    _dev(markov_w1, "markov_w1", _BF16_LIKE)
    _dev(markov_w2, "markov_w2", _BF16_LIKE)
    R = markov_w2.shape[1]
    if markov_w2.shape != (V, R) or markov_w1.shape[1] != R or markov_w1.shape[0] < V:
        raise ValueError("markov_w1 / markov_w2 must be [V, R]")
    _dev(anchor_tokens, "anchor_tokens", (torch.int32,))
    _dev(req_state_idx, "req_state_idx", (torch.int32,))
    _dev(positions, "positions", (torch.int64,))
    _dev(temperature, "temperature", (torch.float32,))
    _dev(seeds, "seeds", (torch.int64, torch.uint64) if hasattr(torch, "uint64") else (torch.int64,))
    _dev(out_tokens, "out_tokens", (torch.int32,))
    S = temperature.shape[0]
    if seeds.shape[0] != S or anchor_tokens.shape[0] != B or req_state_idx.shape[0] != B \
            or positions.shape[0] != B or tuple(out_tokens.shape) != (B, K):
        raise ValueError("inconsistent shapes")
    C = 0
    cache_dt = DSPARK_F32
    if cache is not None:
        _dev(cache, "cache", (torch.float32,) + _BF16_LIKE)
        if cache.dim() != 3 or cache.shape[1] != K or cache.shape[2] != V:
            raise ValueError("cache must be [C, K, V]")
        C = cache.shape[0]
        cache_dt = _logit_dtype(cache, "cache")
    _dev(cache_row_map, "cache_row_map", (torch.int32,))
    need = markov_workspace_bytes(B, K, V, R)
    if workspace_buf is None:
        workspace_buf = workspace(need, base_logits.device)
    _dev(status, "status", (torch.int32,))
    _stats(draft_stats, B, K)
    code = lib().dspark_markov_sample(
        _ptr(base_logits), _logit_dtype(base_logits, "base_logits"), _ptr(markov_w1),
        _ptr(markov_w2), _ptr(anchor_tokens), _ptr(req_state_idx), _ptr(positions),
        _ptr(temperature), _ptr(seeds), _ptr(cache), cache_dt, _ptr(cache_row_map),
        _ptr(out_tokens), _ptr(draft_stats), B, K, V, R, S, max(C, 1), _ptr(workspace_buf),
        workspace_buf.numel() * workspace_buf.element_size(), _ptr(status), _stream(stream))
    _check(code, "dspark_markov_sample")


def markov_sample_wait_limit(base_logits, markov_w1, markov_w2, anchor_tokens, req_state_idx,
                             positions, temperature, seeds, out_tokens, wait_limit_ns,
                             barrier_extra, cache=None, cache_row_map=None, workspace_buf=None,
                             status=None, stream=None):
    """dspark_testing_markov_wait_limit (include/dspark_testing.h): the Markov
    loop with its bounded waits shortened to wait_limit_ns and the grid
    barrier waiting for barrier_extra arrivals more than the grid makes, so
    that a test can make the waits run out."""
    B, K, V = base_logits.shape
    R = markov_w2.shape[1]
    S = temperature.shape[0]
    for t, n in ((base_logits, "base_logits"), (markov_w1, "markov_w1"),
                 (markov_w2, "markov_w2"), (anchor_tokens, "anchor_tokens"),
                 (req_state_idx, "req_state_idx"), (positions, "positions"),
                 (temperature, "temperature"), (seeds, "seeds"), (out_tokens, "out_tokens")):
        _dev(t, n)
    C, cache_dt = 0, DSPARK_F32
    if cache is not None:
        _dev(cache, "cache", (torch.float32,) + _BF16_LIKE)
        C, cache_dt = cache.shape[0], _logit_dtype(cache, "cache")
    if workspace_buf is None:
        workspace_buf = workspace(markov_workspace_bytes(B, K, V, R), base_logits.device)
    _dev(status, "status", (torch.int32,))
    code = lib().dspark_testing_markov_wait_limit(
        _ptr(base_logits), _logit_dtype(base_logits, "base_logits"), _ptr(markov_w1),
        _ptr(markov_w2), _ptr(anchor_tokens), _ptr(req_state_idx), _ptr(positions),
        _ptr(temperature), _ptr(seeds), _ptr(cache), cache_dt, _ptr(cache_row_map),
        _ptr(out_tokens), B, K, V, R, S, max(C, 1), _ptr(workspace_buf),
        workspace_buf.numel() * workspace_buf.element_size(), _ptr(status), _stream(stream),
        int(wait_limit_ns), int(barrier_extra))
    _check(code, "dspark_testing_markov_wait_limit")


# Bytes of the library's fixed scratch array (DSPARK_STATIC_SCRATCH_BYTES).
STATIC_SCRATCH_BYTES = 32 << 10


def markov_sample_static(base_logits, markov_w1, markov_w2, anchor_tokens, req_state_idx,
                         positions, temperature, seeds, out_tokens, cache=None,
                         cache_row_map=None, status=None, stream=None, draft_stats=None):
    """dspark_markov_sample_static on torch tensors: dspark_markov_sample with
    the library's fixed scratch array instead of a workspace, so that nothing
    is allocated (for callers that may not allocate device memory). Calls
    that overlap on the GPU race on that array (see include/dspark.h)."""
    _dev(base_logits, "base_logits", (torch.float32,) + _BF16_LIKE)
    B, K, V = base_logits.shape
    _dev(markov_w1, "markov_w1", _BF16_LIKE)
    _dev(markov_w2, "markov_w2", _BF16_LIKE)
    R = markov_w2.shape[1]
    if markov_w2.shape != (V, R) or markov_w1.shape[1] != R or markov_w1.shape[0] < V:
        raise ValueError("markov_w1 / markov_w2 must be [V, R]")
    for t, n, d in ((anchor_tokens, "anchor_tokens", torch.int32),
                    (req_state_idx, "req_state_idx", torch.int32),
                    (positions, "positions", torch.int64),
                    (temperature, "temperature", torch.float32),
                    (out_tokens, "out_tokens", torch.int32)):
        _dev(t, n, (d,))
    _dev(seeds, "seeds")
    S = temperature.shape[0]
    if seeds.shape[0] != S or anchor_tokens.shape[0] != B or req_state_idx.shape[0] != B \
            or positions.shape[0] != B or tuple(out_tokens.shape) != (B, K):
        raise ValueError("inconsistent shapes")
    C = 0
    cache_dt = DSPARK_F32
    if cache is not None:
        _dev(cache, "cache", (torch.float32,) + _BF16_LIKE)
        if cache.dim() != 3 or cache.shape[1] != K or cache.shape[2] != V:
            raise ValueError("cache must be [C, K, V]")
        C = cache.shape[0]
        cache_dt = _logit_dtype(cache, "cache")
    _dev(cache_row_map, "cache_row_map", (torch.int32,))
    _dev(status, "status", (torch.int32,))
    _stats(draft_stats, B, K)
    code = lib().dspark_markov_sample_static(
        _ptr(base_logits), _logit_dtype(base_logits, "base_logits"), _ptr(markov_w1),
        _ptr(markov_w2), _ptr(anchor_tokens), _ptr(req_state_idx), _ptr(positions),
        _ptr(temperature), _ptr(seeds), _ptr(cache), cache_dt, _ptr(cache_row_map),
        _ptr(out_tokens), _ptr(draft_stats), B, K, V, R, S, max(C, 1), _ptr(status),
        _stream(stream))
    _check(code, "dspark_markov_sample_static")


def markov_sample_topk(base_logits, markov_w1, markov_w2, anchor_tokens, req_state_idx,
                       positions, temperature, seeds, out_tokens, topk, cache=None,
                       cache_row_map=None, workspace_buf=None, status=None, stream=None):
    """dspark_markov_sample_topk on torch tensors: the Markov bias only on the
    top-k base logits of each request and step (see include/dspark.h)."""
    _dev(base_logits, "base_logits", (torch.float32,) + _BF16_LIKE)
    B, K, V = base_logits.shape
    _dev(markov_w1, "markov_w1", _BF16_LIKE)
    _dev(markov_w2, "markov_w2", _BF16_LIKE)
    R = markov_w2.shape[1]
    if markov_w2.shape != (V, R) or markov_w1.shape[1] != R or markov_w1.shape[0] < V:
        raise ValueError("markov_w1 / markov_w2 must be [V, R]")
    for t, n, d in ((anchor_tokens, "anchor_tokens", torch.int32),
                    (req_state_idx, "req_state_idx", torch.int32),
                    (positions, "positions", torch.int64),
                    (temperature, "temperature", torch.float32),
                    (out_tokens, "out_tokens", torch.int32)):
        _dev(t, n, (d,))
    _dev(seeds, "seeds")
    S = temperature.shape[0]
    if seeds.shape[0] != S or anchor_tokens.shape[0] != B or req_state_idx.shape[0] != B \
            or positions.shape[0] != B or tuple(out_tokens.shape) != (B, K):
        raise ValueError("inconsistent shapes")
    C = 0
    cache_dt = DSPARK_F32
    if cache is not None:
        _dev(cache, "cache", (torch.float32,) + _BF16_LIKE)
        if cache.dim() != 3 or cache.shape[1] != K or cache.shape[2] != V:
            raise ValueError("cache must be [C, K, V]")
        C = cache.shape[0]
        cache_dt = _logit_dtype(cache, "cache")
    _dev(cache_row_map, "cache_row_map", (torch.int32,))
    need = int(lib().dspark_markov_topk_workspace_bytes(B, K, V, R, int(topk)))
    if workspace_buf is None:
        workspace_buf = workspace(need, base_logits.device)
    _dev(status, "status", (torch.int32,))
    code = lib().dspark_markov_sample_topk(
        _ptr(base_logits), _logit_dtype(base_logits, "base_logits"), _ptr(markov_w1),
        _ptr(markov_w2), _ptr(anchor_tokens), _ptr(req_state_idx), _ptr(positions),
        _ptr(temperature), _ptr(seeds), _ptr(cache), cache_dt, _ptr(cache_row_map),
        _ptr(out_tokens), int(topk), B, K, V, R, S, max(C, 1), _ptr(workspace_buf),
        workspace_buf.numel() * workspace_buf.element_size(), _ptr(status), _stream(stream))
    _check(code, "dspark_markov_sample_topk")


def rejection_sample(draft_tokens, draft_cache, target_logits, req_state_idx, positions,
                     temperature, top_p, seeds, out_tokens, num_accepted,
                     cache_row_map=None, workspace_buf=None, status=None, stream=None,
                     draft_stats=None):
    """dspark_rejection_sample on torch tensors (see include/dspark.h)."""
    _dev(draft_tokens, "draft_tokens", (torch.int32,))
    B, K = draft_tokens.shape
    _dev(target_logits, "target_logits", (torch.float32,) + _BF16_LIKE)
    if target_logits.dim() != 3 or target_logits.shape[0] != B or target_logits.shape[1] != K + 1:
        raise ValueError("target_logits must be [B, K+1, V]")
    V = target_logits.shape[2]
    C = 0
    cache_dt = DSPARK_F32
    if draft_cache is not None:
        _dev(draft_cache, "draft_cache", (torch.float32,) + _BF16_LIKE)
        if draft_cache.dim() != 3 or draft_cache.shape[1] != K or draft_cache.shape[2] != V:
            raise ValueError("draft_cache must be [C, K, V]")
        C = draft_cache.shape[0]
        cache_dt = _logit_dtype(draft_cache, "draft_cache")
    for t, n, d in ((req_state_idx, "req_state_idx", torch.int32),
                    (positions, "positions", torch.int64),
                    (temperature, "temperature", torch.float32),
                    (top_p, "top_p", torch.float32),
                    (out_tokens, "out_tokens", torch.int32),
                    (num_accepted, "num_accepted", torch.int32)):
        _dev(t, n, (d,))
    _dev(seeds, "seeds")
    S = temperature.shape[0]
    if tuple(out_tokens.shape) != (B, K + 1) or num_accepted.shape[0] != B \
            or top_p.shape[0] != S or seeds.shape[0] != S:
        raise ValueError("inconsistent shapes")
    _dev(cache_row_map, "cache_row_map", (torch.int32,))
    need = verify_workspace_bytes(B, K, V)
    if workspace_buf is None:
        workspace_buf = workspace(need, target_logits.device)
    _dev(status, "status", (torch.int32,))
    _stats(draft_stats, B, K)
    code = lib().dspark_rejection_sample(
        _ptr(draft_tokens), _ptr(draft_cache), cache_dt, _ptr(cache_row_map), _ptr(draft_stats),
        _ptr(target_logits), _logit_dtype(target_logits, "target_logits"),
        _ptr(req_state_idx), _ptr(positions), _ptr(temperature), _ptr(top_p), _ptr(seeds),
        _ptr(out_tokens), _ptr(num_accepted), B, K, V, S, max(C, 1), _ptr(workspace_buf),
        workspace_buf.numel() * workspace_buf.element_size(), _ptr(status), _stream(stream))
    _check(code, "dspark_rejection_sample")


def temperature_divide(z, T, x, stream=None):
    """dspark_testing_temperature_divide on 1-D fp32 device tensors."""
    n = z.numel()
    for t, name in ((z, "z"), (T, "T"), (x, "x")):
        _dev(t, name, (torch.float32,))
        if t.numel() != n:
            raise ValueError("arrays must have equal length")
    _check(lib().dspark_testing_temperature_divide(_ptr(z), _ptr(T), _ptr(x), n,
                                                   _stream(stream)),
           "dspark_testing_temperature_divide")


def noise(seed, pos, col, stream_word, word=None, u=None, g=None, stream=None):
    """dspark_noise on 1-D device tensors of equal length."""
    n = seed.numel()
    for t, name in ((seed, "seed"), (pos, "pos"), (col, "col"), (stream_word, "stream")):
        _dev(t, name)
        if t.numel() != n:
            raise ValueError("noise arrays must have equal length")
    code = lib().dspark_noise(_ptr(seed), _ptr(pos), _ptr(col), _ptr(stream_word),
                              _ptr(word), _ptr(u), _ptr(g), n, _stream(stream))
    _check(code, "dspark_noise")


_PAGED_DTYPES = {torch.bfloat16: DSPARK_BF16, torch.float16: DSPARK_F16,
                 torch.float8_e4m3fn: DSPARK_E4M3}


MAX_PAGED_BATCH = 1024  # DSPARK_MAX_PAGED_BATCH

# The calls below are made once a layer and step, some for a few microseconds of
# work, so their marshalling is kept lean: one pass over a tensor's properties,
# the raw stream handle, one packed struct.
_kv = threading.local()
_KV_FIELDS = struct.Struct("=4Q6q5i")


def _of(t, name, dtype, shape=None):
    """Address of a contiguous CUDA tensor of one dtype (and shape)."""
    try:
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (
                shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _maybe(t, name, dtype, shape=None):
    return None if t is None else _of(t, name, dtype, shape)


def _raw_stream(stream, t):
    """The handle of `stream`, or of the current stream of t's device."""
    return (torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None
            else stream.cuda_stream)


def _rows(t, name):
    """[T, H, D] rows whose tokens may be further apart than H * D (a view into
    a fused projection): (address, dtype, elements between tokens)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dt = t.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise TypeError(f"{name} must be bfloat16 or float16, got {dt}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), _PAGED_DTYPES[dt], H * D if T < 2 else st


def _paged_kv(k_cache, v_cache, k_scale, v_scale):
    """The dspark_paged_kv of caches [num_blocks, kv_heads, page_size, head_dim]
    of any strides with contiguous head_dim (this thread's, until its next call),
    kv_heads and head_dim."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
    dt, shape = k_cache.dtype, k_cache.shape
    if dt is not v_cache.dtype or shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same dtype and shape")
    if dt not in _PAGED_DTYPES:
        raise TypeError(f"k_cache must be bfloat16, float16 or float8_e4m3fn, got {dt}")
    if len(shape) != 4:
        raise ValueError("k_cache must be [num_blocks, kv_heads, page_size, head_dim]")
    N, H, P, D = shape
    kb, kh, kt, kd = k_cache.stride()
    vb, vh, vt, vd = v_cache.stride()
    if (kd != 1 or vd != 1) and D > 1:
        raise ValueError("k_cache and v_cache: the values of a token must be contiguous")
    try:
        kv = _kv.kv
    except AttributeError:
        kv = _kv.kv = PagedKv()
    _KV_FIELDS.pack_into(
        kv, 0, k_cache.data_ptr(), v_cache.data_ptr(),
        0 if k_scale is None else _of(k_scale, "k_scale", torch.float32, (H,)),
        0 if v_scale is None else _of(v_scale, "v_scale", torch.float32, (H,)),
        kb, kh, kt, vb, vh, vt, _PAGED_DTYPES[dt], N, H, P, D)
    return kv, H, D


def paged_tables(req_state_idx, new_lens, cached_lens, block_table, held_blocks, free_blocks,
                 pool, query_start, seq_lens, positions, slot_map, page_size, num_accepted=None,
                 status=None, stream=None):
    """dspark_paged_tables on torch tensors (see include/dspark.h): the step's
    block tables, query offsets, positions and slot map from the request
    lengths; updates cached_lens (with num_accepted), block_table,
    held_blocks, free_blocks and pool."""
    i32, i64 = torch.int32, torch.int64
    B, (S, M) = req_state_idx.shape[0], block_table.shape
    N, T = free_blocks.shape[0], slot_map.shape[0]
    code = (_lib or lib()).dspark_paged_tables(
        _of(req_state_idx, "req_state_idx", i32, (B,)), _of(new_lens, "new_lens", i32, (B,)),
        _of(cached_lens, "cached_lens", i32, (S,)),
        _maybe(num_accepted, "num_accepted", i32, (B,)),
        _of(block_table, "block_table", i32), _of(held_blocks, "held_blocks", i32, (S,)),
        _of(free_blocks, "free_blocks", i32, (N,)), _of(pool, "pool", i32, (2,)),
        _of(query_start, "query_start", i32, (B + 1,)), _of(seq_lens, "seq_lens", i32, (B,)),
        _of(positions, "positions", i64, (T,)), _of(slot_map, "slot_map", i64, (T,)),
        B, S, M, N, T, page_size, _maybe(status, "status", i32),
        _raw_stream(stream, query_start))
    if code:
        _check(code, "dspark_paged_tables")


def kv_append(k, v, k_cache, v_cache, slot_map, k_scale=None, v_scale=None, status=None,
              stream=None):
    """dspark_kv_append on torch tensors (see include/dspark.h): rows k, v
    [T, kv_heads, head_dim] (views of a fused projection will do) into the
    caches [num_blocks, kv_heads, page_size, head_dim]."""
    cache, H, D = _paged_kv(k_cache, v_cache, k_scale, v_scale)
    T = slot_map.shape[0]
    want = (T, H, D)
    kp, dt, ks = _rows(k, "k")
    vp, vdt, vs = _rows(v, "v")
    if k.shape != want or v.shape != want or dt != vdt:
        raise ValueError(f"k and v must be {list(want)} of one dtype")
    code = (_lib or lib()).dspark_kv_append(
        kp, vp, dt, ks, vs, cache, _of(slot_map, "slot_map", torch.int64, (T,)), T,
        _maybe(status, "status", torch.int32), _raw_stream(stream, slot_map))
    if code:
        _check(code, "dspark_kv_append")


def paged_attention_workspace_bytes(B, q_heads, kv_heads, head_dim) -> int:
    return int(lib().dspark_paged_attention_workspace_bytes(B, q_heads, kv_heads, head_dim))


def paged_attention(q, k_cache, v_cache, block_table, req_state_idx, query_start, seq_lens, out,
                    scale=None, causal=True, window=0, k_scale=None, v_scale=None, lse=None,
                    workspace_buf=None, status=None, stream=None):
    """dspark_paged_attention on torch tensors (see include/dspark.h): the
    attention of rows q [T, q_heads, head_dim] (a view of a fused projection
    will do) over the caches, into out and, if given, lse [T, q_heads]. scale
    is 1 / sqrt(head_dim) if not given."""
    cache, H, cd = _paged_kv(k_cache, v_cache, k_scale, v_scale)
    qp, dt, qs = _rows(q, "q")
    T, Hq, D = q.shape
    B, (S, M) = req_state_idx.shape[0], block_table.shape
    if D != cd:
        raise ValueError("q and the caches must have the same head_dim")
    if workspace_buf is None:
        need = paged_attention_workspace_bytes(B, Hq, H, D)
        if stream is None:
            workspace_buf = workspace(need, q.device)
        else:  # memory of the stream that uses it
            with torch.cuda.stream(stream):
                workspace_buf = workspace(need, q.device)
    i32 = torch.int32
    code = (_lib or lib()).dspark_paged_attention(
        qp, dt, qs, cache, _of(block_table, "block_table", i32),
        _of(req_state_idx, "req_state_idx", i32, (B,)),
        _of(query_start, "query_start", i32, (B + 1,)), _of(seq_lens, "seq_lens", i32, (B,)),
        _of(out, "out", q.dtype, q.shape), _maybe(lse, "lse", torch.float32, (T, Hq)),
        D ** -0.5 if scale is None else scale, bool(causal), window, Hq, B, S, M, T,
        workspace_buf.data_ptr(), workspace_buf.nbytes, _maybe(status, "status", i32),
        _raw_stream(stream, q))
    if code:
        _check(code, "dspark_paged_attention")

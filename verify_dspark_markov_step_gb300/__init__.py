"""DSpark Markov drafting step and rejection-sampling verifier on one GB300.

The computation lives in the CUDA library built from ``csrc/`` (C ABI in
``include/dspark.h``); ``_lib`` binds it with ctypes. Submodules:

* ``build``      -- compiles ``_build/libdspark.so`` with nvcc for sm_103a
* ``_lib``       -- the binding (argument marshalling only)
* ``step``       -- one decode step (Markov loop + verification) on device tensors
* ``paged``      -- the paged key/value cache of the verification pass, and a
                    speculative decoding loop on it
* ``rotary``     -- frequencies of rotary positions for the rotating calls
* ``workloads``  -- seeded synthetic inputs
"""

__all__ = ["build", "workloads"]


def __getattr__(name):
    if name in ("markov_sample", "rejection_sample", "noise", "markov_workspace_bytes",
                "verify_workspace_bytes", "status_string", "DsparkError", "lib",
                "paged_tables", "kv_append", "paged_attention",
                "paged_attention_workspace_bytes", "qk_rope", "qk_rope_append",
                "paged_fork", "paged_free", "paged_compact", "paged_compact_workspace_bytes",
                "paged_copy", "PagedCaches"):
        from . import _lib
        globals()[name] = value = getattr(_lib, name)
        return value
    raise AttributeError(name)

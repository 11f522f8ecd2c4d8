"""GB300-native fused row softmax.

``softmax_fwd``, ``attention_fwd`` and the diagnostics beside them are thin ctypes bindings over the
C-ABI library built from ``csrc/``.  The library is loaded on first use, and
its absence is an error, never a fallback.
"""
import importlib

_BINDING_NAMES = frozenset(("softmax_fwd", "softmax_fwd_ptr", "softmax_fwd_masked", "softmax_fwd_masked_ptr",
                            "softmax_fwd_noalloc_ptr", "softmax_fwd_host", "host_workspace_bytes", "attention_fwd",
                            "attention_fwd_ptr", "attention_varlen_fwd", "attention_paged_fwd", "kv_cache_append",
                            "sequence_workspace_bytes", "attention_plan", "set_attention_wait_test", "autotune",
                            "autotune_ptr", "tune_candidates", "autotune_size", "autotune_clear", "plan",
                            "set_force_path", "set_launch_overlap", "last_path", "check_device_error",
                            "set_wait_test", "abi_version", "status_string", "SoftmaxError"))
_binding = None


def __getattr__(name):
    # Asked of the binding every time, so that a function replaced there is the one found
    # here; the module is kept, since importing it anew costs 2 us a call (this, 0.4).
    global _binding
    if name in _BINDING_NAMES:
        if _binding is None:
            _binding = importlib.import_module(".binding", __name__)
        return getattr(_binding, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")

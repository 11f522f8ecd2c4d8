"""GB300-native fused row softmax.

``softmax_fwd``, ``attention_fwd`` and the diagnostics beside them are thin ctypes bindings over the
C-ABI library built from ``csrc/``.  The library is loaded on first use, and
its absence is an error, never a fallback.
"""
import importlib
import types

_BINDING_NAMES = frozenset(("softmax_fwd", "softmax_fwd_ptr", "softmax_fwd_masked", "softmax_fwd_masked_ptr",
                            "softmax_fwd_noalloc_ptr", "softmax_fwd_host", "host_workspace_bytes", "attention_fwd",
                            "attention_fwd_ptr", "attention_varlen_fwd", "attention_paged_fwd", "kv_cache_append",
                            "sequence_workspace_bytes", "attention_plan", "set_attention_wait_test", "autotune",
                            "autotune_ptr", "tune_candidates", "autotune_size", "autotune_clear", "plan",
                            "set_force_path", "set_launch_overlap", "last_path", "check_device_error",
                            "set_wait_test", "abi_version", "status_string", "SoftmaxError"))


class _Binding(types.ModuleType):
    """The binding module: a function replaced in it is the one found in the package from then on."""

    def __setattr__(self, name, value):
        copies = globals()
        if name in _BINDING_NAMES and name in copies and copies[name] is self.__dict__.get(name):
            del copies[name]
        super().__setattr__(name, value)


def __getattr__(name):
    if name in _BINDING_NAMES:
        binding = importlib.import_module(".binding", __name__)
        binding.__class__ = _Binding
        value = getattr(binding, name)
        globals()[name] = value  # the next use finds it without coming here (1 to 2 us a call)
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")

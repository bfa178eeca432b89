"""B200-native fused attention-KL divergence (StreamKL forward and recompute backward).

The compute path is libstreamkl.so (sm_100a kernels behind a C ABI, see
include/streamkl.h); ``streamkl`` is its thin Python binding.

The library is loaded on first use of one of the names below, not on import
of the package: ``attention_kl_distillation_b200.inputs`` and
``attention_kl_distillation_b200.parallel`` carry no CUDA code and can be
imported in a process that must not map the library.
"""
import importlib

_BINDING_NAMES = ("StreamKLError", "bwd", "bwd_algorithm_for", "bwd_noalloc", "fwd", "fwd_splitk",
                  "launch_count", "query_device_status", "set_bwd_algorithm", "set_wait_limit_ms",
                  "splitk_suggest", "splitk_workspace_size", "streamkl", "workspace_size")

_DIFF_NAMES = ("attn_paged", "diff_attn", "diff_attn_bwd", "diff_attn_fwd", "diff_attn_paged",
               "diff_attn_workspace_size", "paged_workspace_size", "paged_write")

__all__ = [*_BINDING_NAMES, *_DIFF_NAMES]


_modules = {}  # a public name's module, once it has been asked for


def __getattr__(name):
    # The name itself is looked up at every use: what is replaced in a module is replaced here.
    module = _modules.get(name)
    if module is None:
        of = ".binding" if name in _BINDING_NAMES else ".diff" if name in _DIFF_NAMES else None
        if of is None:
            raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
        module = _modules[name] = importlib.import_module(of, __name__)
    return getattr(module, name)

"""GB300 block-sparse attention forward: mean-pooled top-k / static block masks
and a tcgen05 block-sparse FlashAttention kernel behind a C ABI (libbsa.so),
the operators around the attention (multi-axis rotary positions, gated norm), and
attention over packed prompts and paged caches of keys and values.

The compute path is the CUDA library only; this package marshals arguments.
The binding (and with it torch) is imported on first use of one of its names, so
that the seeded input generator (``workloads``) can be used without either.
"""
_BINDING_NAMES = (
    "BF16", "FP32", "BsaError", "Index", "StaticSpec", "band_spec", "bsa_build_mask", "bsa_check_device_error",
    "bsa_debug_config", "bsa_forward", "bsa_mask_nnz", "bsa_status_string", "bsa_validate_index",
    "bsa_workspace_size", "build_mask", "cuboid_spec", "explicit_spec", "forward", "load", "workspace")

_BLOCK_NAMES = (
    "GatedNormGrads", "NormSpec", "RotaryPlan", "gated_norm", "gated_norm_backward", "gated_norm_workspace",
    "grid_positions", "rotary", "rotary_backward", "rotary_plan", "rotary_workspace")

_CACHE_NAMES = (
    "KvCache", "cache_attention", "cache_check", "cache_read", "cache_workspace", "cache_write", "kv_cache",
    "prompt_attention")

__all__ = list(_BINDING_NAMES + _BLOCK_NAMES + _CACHE_NAMES)


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    if name in _BLOCK_NAMES:
        from . import block_binding
        value = globals()[name] = getattr(block_binding, name)  # found at once from now on: small calls are bound by the host
        return value
    if name in _CACHE_NAMES:
        from . import cache_binding
        value = globals()[name] = getattr(cache_binding, name)
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")

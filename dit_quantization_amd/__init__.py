"""MI355X-native NVFP4 hot path: block quantizer (absmax / MSE), dequantizer,
W4A16 decode GEMV and W4A4 GEMM as hand-written gfx950 HIP kernels behind a
C ABI (include/nvfp4.h), and beside it the decode path on group-scaled 4-bit
integer weights with 8-bit activations (include/int4.h), 8-bit layers with
block-scaled FP8 weights (include/fp8.h) and paged 8-bit caches of keys and
values (include/kvcache.h).

`dit_quantization_amd.inputs` holds the seeded synthetic workloads.  The
native entry points live in `dit_quantization_amd.nvfp4`, `.int4`, `.fp8` and `.kvcache`, and load
libnvfp4.so on first use; a missing library is an error, never a fallback.
"""
__all__ = ["fp8", "inputs", "int4", "kvcache", "nvfp4"]


def __getattr__(name):
    if name in ("fp8", "int4", "kvcache", "nvfp4"):
        import importlib
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)

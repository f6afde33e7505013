"""MI355X-native FP8 scaled matrix multiply and the operators around it: a
linear layer with its gradient, layer norm with its gradient, quantisation.

The compute runs in the HIP library `libfp8_scaled_mm.so` (built from
`csrc/`); the functions below only marshal torch tensors into the C ABI.
The library is loaded on first use and its absence is an error.
"""
PER_TENSOR = 0
ROWWISE = 1


def __getattr__(name):
    if name in ("fp8_scaled_mm", "fp8_linear", "fp8_linear_backward", "fp8_layer_norm",
                "fp8_layer_norm_backward", "lib", "Fp8MMError", "status_string", "config_names",
                "select_config", "library_path"):
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)

"""BitLinear (W1.58A8) forward for AMD Instinct MI355X (gfx950).

The compute lives in libbitlinear.so (hand-written HIP kernels behind the C
ABI of include/bitlinear.h); ``binding`` marshals torch tensors to it.  The
names below load the library on first use and fail loudly if it is missing.
"""

_EXPORTS = ("pack_weights", "quant_act", "subln_quant_act", "forward", "bitlinear", "linear_grouped",
            "interleave_rows", "gated_relu2", "pack_weights_binary", "forward_binary",
            "gemv_max_tokens",
            "BitLinearError", "load", "last_error")
_EXPERTS = ("Routing", "route_experts", "gated_relu2_experts", "linear_experts")
_W4 = ("pack_weights_w4", "unpack_weights_w4", "forward_w4")


def __getattr__(name):
    if name in _EXPORTS:
        from . import binding                         # looked up every time, as it may be replaced there
        return getattr(binding, name)
    if name in _EXPERTS:
        from . import experts as module
    elif name in _W4:
        from . import w4 as module
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(module, name)   # found at once from now on
    return value

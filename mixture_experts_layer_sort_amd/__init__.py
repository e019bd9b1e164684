"""MI355X (gfx950) dropless top-k Mixture-of-Experts SwiGLU layer.

The layer runs in a HIP library (``libmoe_mi355x.so``, C ABI in
``include/moe.h``); this package holds its ctypes binding (``_lib``), the
buffer-owning runners and autograd functions (``layer``: the layer, the layer
for a few tokens, the residual RMS norm in front of it, and gradient clipping)
and the build script (``build``).
"""
from . import _lib  # noqa: F401
from ._lib import MoEError, lib  # noqa: F401

_LAYER = ("MoELayerRunner", "MoEFunction", "moe_layer", "MoEDecodeRunner", "MoENormRunner", "MoERMSNormFunction",
          "moe_rms_norm", "moe_grad_norm", "moe_clip_grads")

__all__ = ["MoEError", "lib", *_LAYER]


def __getattr__(name):
    if name in _LAYER:
        from . import layer
        return getattr(layer, name)
    raise AttributeError(name)

"""MI355X (gfx950) dropless top-k Mixture-of-Experts SwiGLU layer.

The layer runs in a HIP library (``libmoe_mi355x.so``, C ABI in
``include/moe.h``); this package holds its ctypes binding (``_lib``), the
buffer-owning runners and autograd functions (``layer``: the layer, the layer
for a few tokens, the residual RMS norm in front of it, and gradient clipping;
``mx4``: the layer with experts in 4 bits; ``balance``: the balance loss of
router logits) and the build script (``build``).
"""
from . import _lib  # noqa: F401
from ._lib import MoEError, lib  # noqa: F401

_LAYER = ("MoELayerRunner", "MoEFunction", "moe_layer", "MoEDecodeRunner", "MoENormRunner", "MoERMSNormFunction",
          "moe_rms_norm", "moe_grad_norm", "moe_clip_grads")
_MX4 = ("MoEMx4Tensor", "MoEMx4Runner", "MoEMx4DecodeRunner")
_BALANCE = ("MoEBalanceRunner", "MoEBalanceFunction", "moe_balance_loss")

__all__ = ["MoEError", "lib", *_LAYER, *_MX4, *_BALANCE]


def __getattr__(name):
    if name in _LAYER:
        from . import layer
        return getattr(layer, name)
    if name in _MX4:
        from . import mx4
        return getattr(mx4, name)
    if name in _BALANCE:
        from . import balance
        return getattr(balance, name)
    raise AttributeError(name)

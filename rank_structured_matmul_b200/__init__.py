"""DyRA approximated linear layer for NVIDIA B200 (sm_100a).

The compute runs in libdyra.so (hand-written CUDA: tcgen05/TMA kernels for
bf16, SIMT kernels for fp32) behind the C ABI of include/dyra.h; `dyra` is
its ctypes binding and `prep` the host-side offline preparation. `layers` binds
the exact layers beside it (include/dyra_layers.h): a dense layer with its
epilogue and gradients, and a mixture-of-experts layer for a few tokens.
"""

from . import dyra, layers, prep  # noqa: F401
from .dyra import DyraError, DyraLinear  # noqa: F401
from .layers import DenseLinear, MoeLayer  # noqa: F401

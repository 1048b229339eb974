"""Exact layers beside the approximated one (include/dyra_layers.h).

DenseLinear: a dense linear layer with bias, activation and residual in its
epilogue, and its gradients. MoeLayer: a mixture-of-experts layer for a few
tokens. As in dyra.py this marshals arguments only; every step runs in
libdyra.so's CUDA kernels and there is no fallback.

Weights are arguments of each call. Tensors are contiguous CUDA tensors of the
layer's type on the layer's device (the current device when it was made); a
call runs on `stream` (default: that device's current stream), where its
results are allocated too. Torch records no gradient of these calls (the dense
layer's are DenseLinear.backward's): where it would have to, the call is refused.
"""

from __future__ import annotations

import ctypes
import operator

from .dyra import DYRA_BF16, DYRA_ERR_INVALID_ARG, DYRA_F32, DyraError, _check, _ptr, lib

DYRA_ACT_NONE = 0
DYRA_ACT_RELU = 1
DYRA_ACT_GELU = 2
DYRA_ACT_GELU_TANH = 3
DYRA_ACT_SILU = 4
ACTIVATIONS = {"none": DYRA_ACT_NONE, "relu": DYRA_ACT_RELU, "gelu": DYRA_ACT_GELU,
               "gelu_tanh": DYRA_ACT_GELU_TANH, "silu": DYRA_ACT_SILU}

DYRA_MOE_MAX_TOP_K = 16
DYRA_MOE_MAX_EXPERTS = 512


# ---- raw C-ABI wrappers (same names; ints or tensors for pointers) ----

def _c_ints(where: str, *values) -> None:
    """Values that a C int does not hold are refused like other sizes out of range
    (ctypes would pass their low 32 bits)."""
    for v in values:
        if not -2 ** 31 <= operator.index(v) < 2 ** 31:
            raise DyraError(DYRA_ERR_INVALID_ARG, where)


def dyra_dense_create(d_in: int, d_out: int, dtype: int) -> int:
    _c_ints("dyra_dense_create", d_in, d_out, dtype)
    h = ctypes.c_void_p()
    _check(lib().dyra_dense_create(ctypes.byref(h), d_in, d_out, dtype), "dyra_dense_create")
    return h.value


def dyra_dense_forward(p: int, X, W, bias, residual, act: int, Y, Z, N: int, stream) -> None:
    _check(lib().dyra_dense_forward(p, _ptr(X), _ptr(W), _ptr(bias), _ptr(residual), act, _ptr(Y),
                                    _ptr(Z), N, stream), "dyra_dense_forward")


def dyra_dense_backward(p: int, dY, X, W, Z, act: int, dZ, dX, dW, dbias, N: int, stream) -> None:
    _check(lib().dyra_dense_backward(p, _ptr(dY), _ptr(X), _ptr(W), _ptr(Z), act, _ptr(dZ),
                                     _ptr(dX), _ptr(dW), _ptr(dbias), N, stream),
           "dyra_dense_backward")


def dyra_dense_status(p: int) -> int:
    return _check(lib().dyra_dense_status(p), "dyra_dense_status")


def dyra_dense_device_bytes(p: int) -> int:
    return int(lib().dyra_dense_device_bytes(p))


def dyra_dense_destroy(p: int) -> None:
    _check(lib().dyra_dense_destroy(p), "dyra_dense_destroy")


def dyra_moe_create(d_model: int, d_ff: int, experts: int, top_k: int, act: int, renorm: int,
                    dtype: int) -> int:
    _c_ints("dyra_moe_create", d_model, d_ff, experts, top_k, act, renorm, dtype)
    h = ctypes.c_void_p()
    _check(lib().dyra_moe_create(ctypes.byref(h), d_model, d_ff, experts, top_k, act, renorm,
                                 dtype), "dyra_moe_create")
    return h.value


def dyra_moe_route(p: int, X, Wr, ids, weights, N: int, stream) -> None:
    _check(lib().dyra_moe_route(p, _ptr(X), _ptr(Wr), _ptr(ids), _ptr(weights), N, stream),
           "dyra_moe_route")


def dyra_moe_experts(p: int, X, ids, weights, Wgu, Wd, residual, Y, N: int, stream) -> None:
    _check(lib().dyra_moe_experts(p, _ptr(X), _ptr(ids), _ptr(weights), _ptr(Wgu), _ptr(Wd),
                                  _ptr(residual), _ptr(Y), N, stream), "dyra_moe_experts")


def dyra_moe_forward(p: int, X, Wr, Wgu, Wd, residual, Y, ids, weights, N: int, stream) -> None:
    _check(lib().dyra_moe_forward(p, _ptr(X), _ptr(Wr), _ptr(Wgu), _ptr(Wd), _ptr(residual),
                                  _ptr(Y), _ptr(ids), _ptr(weights), N, stream),
           "dyra_moe_forward")


def dyra_moe_status(p: int) -> int:
    return _check(lib().dyra_moe_status(p), "dyra_moe_status")


def dyra_moe_device_bytes(p: int) -> int:
    return int(lib().dyra_moe_device_bytes(p))


def dyra_moe_destroy(p: int) -> None:
    _check(lib().dyra_moe_destroy(p), "dyra_moe_destroy")


def dyra_debug_dense_set_wait_limit(p: int, ns: int) -> None:
    _check(lib().dyra_debug_dense_set_wait_limit(p, ns), "dyra_debug_dense_set_wait_limit")


def dyra_debug_moe_set_wait_limit(p: int, ns: int) -> None:
    _check(lib().dyra_debug_moe_set_wait_limit(p, ns), "dyra_debug_moe_set_wait_limit")


# ---- convenience objects ----

def _activation(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, not %r" % (", ".join(ACTIVATIONS), act))
    return code


class _Layer:
    """What both layers share: type, device, checks of tensors, streams. A call of
    a few microseconds' work is bound by what runs here, so the checks are single
    comparisons and the current stream is read without an object for it."""

    def _setup(self, dtype: str) -> int:
        import torch
        if dtype not in ("bf16", "f32"):
            raise ValueError("dtype must be 'bf16' or 'f32', not %r" % (dtype,))
        self.dtype = dtype
        self.torch_dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.int32, self.float32 = torch.int32, torch.float32
        self._recording = torch.is_grad_enabled
        self.handle = None
        return DYRA_BF16 if dtype == "bf16" else DYRA_F32

    def _bind(self, handle: int) -> None:
        import torch
        self.handle = handle
        self.index = torch.cuda.current_device()
        self.device = torch.device("cuda", self.index)
        self._raw_stream = torch._C._cuda_getCurrentRawStream

    def _need(self, name, t, shape, dtype=None):
        """A contiguous tensor of the shape and type on the layer's device."""
        if t is None or t.shape != shape or t.dtype is not (dtype or self.torch_dtype) \
                or t.get_device() != self.index or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                             % (name, dtype or self.torch_dtype, tuple(shape), self.device))
        if t.requires_grad and self._recording():  # the results would come without one
            raise ValueError("%s requires a gradient, and torch records none of this call: make "
                             "it under torch.no_grad() or with detached tensors" % name)

    def _rows(self, X, width, name="X"):
        if X is None or X.dim() != 2:
            raise ValueError("%s must be a matrix of %d columns" % (name, width))
        N = X.shape[0]
        self._need(name, X, (N, width))
        return N

    def _on(self, stream):
        """(stream object to allocate on, or None for the current one; cudaStream_t)"""
        if stream is None:
            return None, self._raw_stream(self.index)
        if isinstance(stream, int):
            import torch
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        return stream, stream.cuda_stream

    def _new(self, like, on, *shapes):
        """New tensors of the layer's type (None for a shape of None), allocated on
        the call's stream. (Sizes as arguments: as one tuple they take new_empty half
        as long again, 1.9 us instead of 1.4.)"""
        if on is not None:
            import torch
            with torch.cuda.stream(on):
                return self._new(like, None, *shapes)
        new = like.new_empty
        return [new(*s) if s else None for s in shapes]

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DenseLinear(_Layer):
    """One dense linear layer shape on the current CUDA device."""

    def __init__(self, d_in: int, d_out: int, dtype: str = "bf16"):
        code = self._setup(dtype)
        self.d_in, self.d_out = d_in, d_out
        self._bind(dyra_dense_create(d_in, d_out, code))

    def forward(self, X, W, bias=None, residual=None, act: str = "none", save_z: bool = False,
                Y=None, stream=None):
        """Y = act(X W^T + bias) + residual; with save_z the pair (Y, Z), Z the
        pre-activations that backward() takes. Y may be given, and may be the
        residual itself."""
        code = _activation(act)
        N = self._rows(X, self.d_in)
        out = (N, self.d_out)
        self._need("W", W, (self.d_out, self.d_in))
        if bias is not None:
            self._need("bias", bias, (self.d_out,))
        if residual is not None:
            self._need("residual", residual, out)
        if Y is not None:
            self._need("Y", Y, out)
        on, s = self._on(stream)
        new, Z = self._new(X, on, None if Y is not None else out, out if save_z else None)
        Y = new if Y is None else Y
        dyra_dense_forward(self.handle, X, W, bias, residual, code, Y, Z, N, s)
        return (Y, Z) if save_z else Y

    def backward(self, dY, X, W, Z=None, act: str = "none", need_dX: bool = True,
                 need_dW: bool = True, need_dbias: bool = True, stream=None):
        """(dX, dW, dbias) from dY (None where not needed); the gradient of the
        residual is dY. Z: the forward's pre-activations, unless act is 'none'.
        X is not read without dW, W not without dX."""
        code = _activation(act)
        N = self._rows(dY, self.d_out, "dY")
        if need_dW or X is not None:
            self._need("X", X, (N, self.d_in))
        if need_dX or W is not None:
            self._need("W", W, (self.d_out, self.d_in))
        if code != DYRA_ACT_NONE:
            self._need("Z", Z, (N, self.d_out))
        on, s = self._on(stream)
        # dZ is freed on return: the allocator hands it out again in stream order
        dX, dW, dbias, dZ = self._new(
            dY, on, (N, self.d_in) if need_dX else None,
            (self.d_out, self.d_in) if need_dW else None, (self.d_out,) if need_dbias else None,
            (N, self.d_out) if code != DYRA_ACT_NONE else None)
        dyra_dense_backward(self.handle, dY, X, W, Z, code, dZ, dX, dW, dbias, N, s)
        return dX, dW, dbias

    def status(self) -> int:
        return dyra_dense_status(self.handle)

    def device_bytes(self) -> int:
        return dyra_dense_device_bytes(self.handle)

    def close(self) -> None:
        if self.handle:
            dyra_dense_destroy(self.handle)
            self.handle = None


class MoeLayer(_Layer):
    """One mixture-of-experts layer shape on the current CUDA device: gated
    experts d_model -> d_ff -> d_model, top_k of them per token."""

    def __init__(self, d_model: int, d_ff: int, experts: int, top_k: int, dtype: str = "bf16",
                 act: str = "silu", renorm: bool = True):
        code = self._setup(dtype)
        self.d_model, self.d_ff, self.experts_n, self.top_k = d_model, d_ff, experts, top_k
        self._bind(dyra_moe_create(d_model, d_ff, experts, top_k, _activation(act),
                                   int(bool(renorm)), code))

    def _need_experts(self, X, Wgu, Wd, residual, Y):
        N = self._rows(X, self.d_model)
        self._need("Wgu", Wgu, (self.experts_n, 2 * self.d_ff, self.d_model))
        self._need("Wd", Wd, (self.experts_n, self.d_model, self.d_ff))
        if residual is not None:
            self._need("residual", residual, (N, self.d_model))
        if Y is not None:
            self._need("Y", Y, (N, self.d_model))
        return N

    def _new_routing(self, X, on, N):
        if on is not None:
            import torch
            with torch.cuda.stream(on):
                return self._new_routing(X, None, N)
        return (X.new_empty(N, self.top_k, dtype=self.int32),
                X.new_empty(N, self.top_k, dtype=self.float32))

    def route(self, X, Wr, stream=None):
        """(ids, weights): each token's top_k experts, largest logit first (the
        lower index among equals), and their softmax weights."""
        N = self._rows(X, self.d_model)
        self._need("Wr", Wr, (self.experts_n, self.d_model))
        on, s = self._on(stream)
        ids, weights = self._new_routing(X, on, N)
        dyra_moe_route(self.handle, X, Wr, ids, weights, N, s)
        return ids, weights

    def experts(self, X, ids, weights, Wgu, Wd, residual=None, Y=None, stream=None):
        """sum over k of weights[n][k] * expert ids[n][k] of token n, + residual.
        Ids outside the experts (such as -1) add nothing."""
        N = self._need_experts(X, Wgu, Wd, residual, Y)
        self._need("ids", ids, (N, self.top_k), self.int32)
        self._need("weights", weights, (N, self.top_k), self.float32)
        on, s = self._on(stream)
        if Y is None:
            Y, = self._new(X, on, (N, self.d_model))
        dyra_moe_experts(self.handle, X, ids, weights, Wgu, Wd, residual, Y, N, s)
        return Y

    def forward(self, X, Wr, Wgu, Wd, residual=None, Y=None, stream=None):
        """The whole layer: (Y, ids, weights)."""
        N = self._need_experts(X, Wgu, Wd, residual, Y)
        self._need("Wr", Wr, (self.experts_n, self.d_model))
        on, s = self._on(stream)
        ids, weights = self._new_routing(X, on, N)
        if Y is None:
            Y, = self._new(X, on, (N, self.d_model))
        dyra_moe_forward(self.handle, X, Wr, Wgu, Wd, residual, Y, ids, weights, N, s)
        return Y, ids, weights

    def status(self) -> int:
        return dyra_moe_status(self.handle)

    def device_bytes(self) -> int:
        return dyra_moe_device_bytes(self.handle)

    def close(self) -> None:
        if self.handle:
            dyra_moe_destroy(self.handle)
            self.handle = None

"""Python binding of include/mlp_block.h: layer norm, and the linear operator with bias, activation and
residual in its epilogue, dense or grouped by expert, forward and backward.

Argument checks and marshalling only, compiled (csrc/marshal.cpp) because a call takes a few microseconds: every
tensor is a CUDA tensor of the caller's, outputs and workspaces included, all of a call on one device (x's for layer
norm, the handle's for Linear), and a call enqueues work on ``stream`` (default: torch's current stream of that device)
without synchronising.  A wrong dtype, shape, device or order of elements raises ValueError, an error of the library
(strides and alignments that it does not take, for instance) MlpChainError.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import LinearDesc, LinearPlan
from .chain import DT_BF16, DT_F32, MlpChainError, _check

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
_DTYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


_marshal = None


def _load():
    global _marshal
    _marshal = _lib.load_marshal()
    return _marshal


# -------------------------------------------------------------------------------- layer norm --
def layer_norm_forward(x, gamma, beta, y, *, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """y = (x - mean) rstd * gamma + beta over the rows of x (mlp_layernorm_forward).  gamma and beta may be
    None; mean and rstd (float32 [rows], kept for the backward pass) are optional; y may be x."""
    status = (_marshal or _load()).norm_forward(x, gamma, beta, y, mean, rstd, eps, stream)
    if status:
        raise MlpChainError(status, "mlp_layernorm_forward")


@functools.lru_cache(maxsize=1024)
def layer_norm_workspace_size(rows: int, cols: int) -> int:
    """Bytes of workspace of layer_norm_backward with dgamma or dbeta."""
    n = ctypes.c_size_t()
    _check(_lib.load().mlp_layernorm_workspace_size(rows, cols, ctypes.byref(n)), "mlp_layernorm_workspace_size")
    return n.value


def layer_norm_backward(dy, x, gamma, mean, rstd, dx, *, dgamma=None, dbeta=None, dx_add=None, workspace=None,
                        stream=None):
    """Gradients of layer_norm_forward (mlp_layernorm_backward): dx (plus dx_add, the gradient that arrives by
    another path), dgamma and dbeta, each optional."""
    status = (_marshal or _load()).norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dx_add, workspace, stream)
    if status:
        raise MlpChainError(status, "mlp_layernorm_backward")


# ------------------------------------------------------------------------------------ linear --
class Linear:
    """Y = act(X W + b) + R and its gradients (mlp_linear): a handle fixes K, N, the activation ("none", "relu",
    "gelu" (tanh form), "silu"), the weight layout ("kn" or "nk") and the number of experts; the number of
    rows may differ from call to call.

    experts=0: W is [K, N] ("kn") or [N, K] ("nk"), bias [N].  experts=E: W and bias have a leading dimension E,
    and every call takes ``offsets`` (int32 [E + 1] on the device): rows offsets[e] .. offsets[e+1] belong to
    expert e.  X, Y, Z, residual and their gradients are bfloat16 matrices, possibly slices of wider ones (row
    strides in multiples of 8 elements).
    """

    def __init__(self, K: int, N: int, *, activation: Optional[str] = None, experts: int = 0, weight_layout: str = "kn",
                 bias_dtype=torch.bfloat16, dw_dtype=torch.bfloat16, device: int = 0, timeout_us: int = 0):
        self._h = self._args = None
        lib, marshal = _lib.load(), _marshal or _load()
        activation = activation or "none"
        if activation not in ACTIVATIONS or weight_layout not in ("kn", "nk"):
            raise ValueError(f"unknown activation {activation!r} or weight layout {weight_layout!r}")
        if bias_dtype not in _DTYPES or dw_dtype not in _DTYPES:
            raise ValueError("bias_dtype and dw_dtype are bfloat16 or float32")
        d = LinearDesc(K, N, experts, 0 if weight_layout == "kn" else 1, ACTIVATIONS[activation], _DTYPES[bias_dtype],
                       _DTYPES[dw_dtype], device, timeout_us)
        h = ctypes.c_void_p()
        _check(lib.mlp_linear_create(ctypes.byref(d), ctypes.byref(h)), "mlp_linear_create")
        self._lib, self._h = lib, h
        self._args = marshal.linear(h.value, int(K), int(N), int(experts), d.weight_layout, d.activation, d.bias_dtype,
                                    d.dw_dtype, int(device))
        self.K, self.N, self.experts, self.activation = int(K), int(N), int(experts), activation
        self.bias_dtype, self.dw_dtype, self.device = bias_dtype, dw_dtype, int(device)
        lead = (self.experts,) if self.experts else ()
        self.weight_shape = lead + ((self.K, self.N) if weight_layout == "kn" else (self.N, self.K))
        self.bias_shape = lead + (self.N,)

    def close(self):
        if self._h:
            self._lib.mlp_linear_destroy(self._h)
            self._h = self._args = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def workspace_size(self, rows: int) -> int:
        """Bytes of workspace backward() needs for this many rows (forward() needs none)."""
        n = ctypes.c_size_t()
        _check(self._lib.mlp_linear_workspace_size(self._h, rows, ctypes.byref(n)), "mlp_linear_workspace_size")
        return n.value

    def forward(self, X, W, Y, *, bias=None, residual=None, Z=None, offsets=None, workspace=None, stream=None):
        """Y = act(X W + bias) + residual; Z (optional) receives the pre-activation X W + bias.  workspace is
        accepted for symmetry with backward() and not used."""
        status = _marshal.linear_forward(self._args, X, W, Y, bias, residual, Z, offsets, stream)
        if status:
            raise MlpChainError(status, "mlp_linear_forward")

    def backward(self, dY, X, W, *, Z=None, dX=None, dW=None, dbias=None, offsets=None, workspace=None, stream=None):
        """The gradients asked for, of forward() at pre-activation Z (not needed without an activation).  X may be
        None without dW, W without dX.  The residual's gradient is dY itself."""
        status = _marshal.linear_backward(self._args, dY, X, W, Z, dX, dW, dbias, offsets, workspace, stream)
        if status:
            raise MlpChainError(status, "mlp_linear_backward")

    def check(self, stream=None) -> int:
        """Synchronise and return the device status (0 = OK); clears it."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        return int(self._lib.mlp_linear_check(self._h, (stream if isinstance(stream, int) else stream.cuda_stream) or None))

    def plan(self, rows: int, what: str = "Y") -> dict:
        """The kernel variant that computes "Y", "dX" or "dW" for this many rows."""
        p = LinearPlan()
        _check(self._lib.mlp_linear_get_plan(self._h, rows, ("Y", "dX", "dW").index(what), ctypes.byref(p)),
               "mlp_linear_get_plan")
        return {"form": ("rows", "rows_t", "reduce")[p.form], "cta_pair": p.cta_pair, "tile_cols": p.tile_cols,
                "k_split": p.k_split, "pipe_stages": p.pipe_stages}

"""Python binding of include/mlp_block.h: layer norm, and the linear operator with bias, activation and
residual in its epilogue, dense or grouped by expert, forward and backward.

Argument checks and marshalling only: every tensor is a CUDA tensor of the caller's, outputs and
workspaces included, and a call enqueues work on ``stream`` (default: torch's current stream) without
synchronising.  A wrong dtype, shape or stride raises ValueError, an error of the library MlpChainError.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import LinearDesc, LinearPlan
from .chain import DT_BF16, DT_F32, _check

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
_DTYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _matrix(t, name, rows, cols, dtype, optional=True):
    """(address, row stride) of a rows x cols matrix with contiguous rows."""
    if t is None:
        if optional:
            return None, 0
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor {dtype} [{rows}, {cols}], got {t.dtype} {list(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.data_ptr(), (s0 if rows > 1 else max(cols, s0))


def _dense(t, name, shape, dtype, optional=True):
    """Address of a contiguous tensor of this shape."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or tuple(t.shape) != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _workspace(t, need, name="workspace"):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < need:
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of at least {need} bytes")
    return t.data_ptr()


# -------------------------------------------------------------------------------- layer norm --
def _norm_types(x, gamma, *more):
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError("layer norm takes matrices of bfloat16 or float32")
    wd = next((w.dtype for w in (gamma, *more) if w is not None), torch.float32)
    if wd not in _DTYPES:
        raise ValueError("layer norm weights are bfloat16 or float32")
    return x.shape[0], x.shape[1], wd


def layer_norm_forward(x, gamma, beta, y, *, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """y = (x - mean) rstd * gamma + beta over the rows of x (mlp_layernorm_forward).  gamma and beta may be
    None; mean and rstd (float32 [rows], kept for the backward pass) are optional; y may be x."""
    lib = _lib.load()
    R, C, wd = _norm_types(x, gamma, beta)
    px, ldx = _matrix(x, "x", R, C, x.dtype)
    py, ldy = _matrix(y, "y", R, C, x.dtype, optional=False)
    _check(lib.mlp_layernorm_forward(R, C, px, ldx, _DTYPES[x.dtype], _dense(gamma, "gamma", (C,), wd),
                                     _dense(beta, "beta", (C,), wd), _DTYPES[wd], eps, py, ldy,
                                     _dense(mean, "mean", (R,), torch.float32),
                                     _dense(rstd, "rstd", (R,), torch.float32), _stream(stream)),
           "mlp_layernorm_forward")


def layer_norm_workspace_size(rows: int, cols: int) -> int:
    """Bytes of workspace of layer_norm_backward with dgamma or dbeta."""
    n = ctypes.c_size_t()
    _check(_lib.load().mlp_layernorm_workspace_size(rows, cols, ctypes.byref(n)), "mlp_layernorm_workspace_size")
    return n.value


def layer_norm_backward(dy, x, gamma, mean, rstd, dx, *, dgamma=None, dbeta=None, dx_add=None, workspace=None,
                        stream=None):
    """Gradients of layer_norm_forward (mlp_layernorm_backward): dx (plus dx_add, the gradient that arrives by
    another path), dgamma and dbeta, each optional."""
    lib = _lib.load()
    R, C, wd = _norm_types(x, gamma, dgamma, dbeta)
    pdy, lddy = _matrix(dy, "dy", R, C, x.dtype, optional=False)
    px, ldx = _matrix(x, "x", R, C, x.dtype)
    pa, lda = _matrix(dx_add, "dx_add", R, C, x.dtype)
    pdx, lddx = _matrix(dx, "dx", R, C, x.dtype)
    need = layer_norm_workspace_size(R, C) if dgamma is not None or dbeta is not None else 0
    _check(lib.mlp_layernorm_backward(R, C, pdy, lddy, px, ldx, _DTYPES[x.dtype], _dense(gamma, "gamma", (C,), wd),
                                      _DTYPES[wd], _dense(mean, "mean", (R,), torch.float32, optional=False),
                                      _dense(rstd, "rstd", (R,), torch.float32, optional=False), pa, lda, pdx, lddx,
                                      _dense(dgamma, "dgamma", (C,), wd), _dense(dbeta, "dbeta", (C,), wd),
                                      _workspace(workspace, need), _stream(stream)), "mlp_layernorm_backward")


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
        self._h = None
        lib = _lib.load()
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
        self.K, self.N, self.experts, self.activation = int(K), int(N), int(experts), activation
        self.bias_dtype, self.dw_dtype = bias_dtype, dw_dtype
        lead = (self.experts,) if self.experts else ()
        self.weight_shape = lead + ((self.K, self.N) if weight_layout == "kn" else (self.N, self.K))
        self.bias_shape = lead + (self.N,)

    def close(self):
        if self._h:
            self._lib.mlp_linear_destroy(self._h)
            self._h = None

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

    def _offsets(self, t):
        if not self.experts:
            if t is not None:
                raise ValueError("offsets: this handle has no experts")
            return None
        return _dense(t, "offsets", (self.experts + 1,), torch.int32, optional=False)

    def forward(self, X, W, Y, *, bias=None, residual=None, Z=None, offsets=None, workspace=None, stream=None):
        """Y = act(X W + bias) + residual; Z (optional) receives the pre-activation X W + bias.  workspace is
        accepted for symmetry with backward() and not used."""
        R = X.shape[0]
        bf = torch.bfloat16
        px, ldx = _matrix(X, "X", R, self.K, bf)
        py, ldy = _matrix(Y, "Y", R, self.N, bf, optional=False)
        pr, ldr = _matrix(residual, "residual", R, self.N, bf)
        pz, ldz = _matrix(Z, "Z", R, self.N, bf)
        _check(self._lib.mlp_linear_forward(self._h, R, px, ldx, _dense(W, "W", self.weight_shape, bf, optional=False),
                                            _dense(bias, "bias", self.bias_shape, self.bias_dtype), pr, ldr,
                                            self._offsets(offsets), pz, ldz, py, ldy, _stream(stream)),
               "mlp_linear_forward")

    def backward(self, dY, X, W, *, Z=None, dX=None, dW=None, dbias=None, offsets=None, workspace=None, stream=None):
        """The gradients asked for, of forward() at pre-activation Z (not needed without an activation).  X may be
        None without dW, W without dX.  The residual's gradient is dY itself."""
        R = dY.shape[0]
        bf = torch.bfloat16
        pdy, lddy = _matrix(dY, "dY", R, self.N, bf)
        px, ldx = _matrix(X, "X", R, self.K, bf, optional=dW is None)
        pz, ldz = _matrix(Z, "Z", R, self.N, bf, optional=self.activation == "none")
        pdx, lddx = _matrix(dX, "dX", R, self.K, bf)
        need = self.workspace_size(R) if dbias is not None or self.activation != "none" else 0
        _check(self._lib.mlp_linear_backward(self._h, R, pdy, lddy, px, ldx,
                                             _dense(W, "W", self.weight_shape, bf, optional=dX is None), pz, ldz,
                                             self._offsets(offsets), pdx, lddx,
                                             _dense(dW, "dW", self.weight_shape, self.dw_dtype),
                                             _dense(dbias, "dbias", self.bias_shape, self.bias_dtype),
                                             _workspace(workspace, need), _stream(stream)), "mlp_linear_backward")

    def check(self, stream=None) -> int:
        """Synchronise and return the device status (0 = OK); clears it."""
        return int(self._lib.mlp_linear_check(self._h, _stream(stream)))

    def plan(self, rows: int, what: str = "Y") -> dict:
        """The kernel variant that computes "Y", "dX" or "dW" for this many rows."""
        p = LinearPlan()
        _check(self._lib.mlp_linear_get_plan(self._h, rows, ("Y", "dX", "dW").index(what), ctypes.byref(p)),
               "mlp_linear_get_plan")
        return {"form": ("rows", "rows_t", "reduce")[p.form], "cta_pair": p.cta_pair, "tile_cols": p.tile_cols,
                "k_split": p.k_split, "pipe_stages": p.pipe_stages}

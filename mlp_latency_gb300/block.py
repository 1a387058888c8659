"""Python binding of include/mlp_block.h: layer norm, and the linear operator with bias, activation and
residual in its epilogue, dense or grouped by expert, forward and backward.

Argument checks and marshalling only: every tensor is a CUDA tensor of the caller's, outputs and
workspaces included, and a call enqueues work on ``stream`` (default: torch's current stream) without
synchronising.  A wrong dtype, shape or stride raises ValueError, an error of the library MlpChainError.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import LinearDesc, LinearPlan
from .chain import DT_BF16, DT_F32, _check

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
_DTYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


def _stream(stream, device: int) -> Optional[int]:
    if stream is None:   # torch.cuda.current_stream(device).cuda_stream without the 3 us of building the object
        return torch._C._cuda_getCurrentRawStream(device) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _matrix(t, name, shape, dtype):
    """(address, row stride) of a matrix with contiguous rows.  (These checks run on every call of a few
    microseconds, so they touch each tensor as few times as they can.)"""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor {dtype} {list(shape)}, got {t.dtype} {list(t.shape)} on {t.device}")
    ld, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1] + 7 & -8)   # (one row: any stride will do)


def _dense(t, name, shape, dtype):
    """Address of a contiguous tensor of this shape."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor {dtype} {list(shape)}, got {t.dtype} {list(t.shape)} "
                         f"on {t.device}")
    return t.data_ptr()


def _workspace(t, need):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < need:
        raise ValueError(f"workspace: expected a contiguous CUDA tensor of at least {need} bytes")
    return t.data_ptr()


# -------------------------------------------------------------------------------- layer norm --
def _norm_types(x, *weights):
    shape, dt = x.shape, _DTYPES.get(x.dtype)
    if len(shape) != 2 or dt is None:
        raise ValueError("layer norm takes matrices of bfloat16 or float32")
    for w in weights:
        if w is not None:
            wd = w.dtype
            if wd not in _DTYPES:
                raise ValueError("layer norm weights are bfloat16 or float32")
            return shape, dt, wd
    return shape, dt, torch.float32


def layer_norm_forward(x, gamma, beta, y, *, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """y = (x - mean) rstd * gamma + beta over the rows of x (mlp_layernorm_forward).  gamma and beta may be
    None; mean and rstd (float32 [rows], kept for the backward pass) are optional; y may be x."""
    shape, dt, wd = _norm_types(x, gamma, beta)
    R, C = shape
    px, ldx = _matrix(x, "x", shape, x.dtype)
    py, ldy = _matrix(y, "y", shape, x.dtype)
    _check(_lib.load().mlp_layernorm_forward(
        R, C, px, ldx, dt, None if gamma is None else _dense(gamma, "gamma", (C,), wd),
        None if beta is None else _dense(beta, "beta", (C,), wd), _DTYPES[wd], eps, py, ldy,
        None if mean is None else _dense(mean, "mean", (R,), torch.float32),
        None if rstd is None else _dense(rstd, "rstd", (R,), torch.float32), _stream(stream, x.get_device())),
        "mlp_layernorm_forward")


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
    shape, dt, wd = _norm_types(x, gamma, dgamma, dbeta)
    R, C = shape
    xd = x.dtype
    pdy, lddy = _matrix(dy, "dy", shape, xd)
    px, ldx = _matrix(x, "x", shape, xd)
    pa, lda = (None, 0) if dx_add is None else _matrix(dx_add, "dx_add", shape, xd)
    pdx, lddx = (None, 0) if dx is None else _matrix(dx, "dx", shape, xd)
    need = layer_norm_workspace_size(R, C) if dgamma is not None or dbeta is not None else 0
    _check(_lib.load().mlp_layernorm_backward(
        R, C, pdy, lddy, px, ldx, dt, None if gamma is None else _dense(gamma, "gamma", (C,), wd), _DTYPES[wd],
        _dense(mean, "mean", (R,), torch.float32), _dense(rstd, "rstd", (R,), torch.float32), pa, lda, pdx, lddx,
        None if dgamma is None else _dense(dgamma, "dgamma", (C,), wd),
        None if dbeta is None else _dense(dbeta, "dbeta", (C,), wd), _workspace(workspace, need),
        _stream(stream, x.get_device())), "mlp_layernorm_backward")


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
        self._lib, self._h, self._ws_sizes = lib, h, {}
        self.K, self.N, self.experts, self.activation = int(K), int(N), int(experts), activation
        self.bias_dtype, self.dw_dtype, self.device = bias_dtype, dw_dtype, int(device)
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
        need = self._ws_sizes.get(rows)
        if need is None:
            n = ctypes.c_size_t()
            _check(self._lib.mlp_linear_workspace_size(self._h, rows, ctypes.byref(n)), "mlp_linear_workspace_size")
            need = self._ws_sizes[rows] = n.value
        return need

    def _offsets(self, t):
        if not self.experts:
            if t is not None:
                raise ValueError("offsets: this handle has no experts")
            return None
        return _dense(t, "offsets", (self.experts + 1,), torch.int32)

    def forward(self, X, W, Y, *, bias=None, residual=None, Z=None, offsets=None, workspace=None, stream=None):
        """Y = act(X W + bias) + residual; Z (optional) receives the pre-activation X W + bias.  workspace is
        accepted for symmetry with backward() and not used."""
        R = X.shape[0]
        bf, out = torch.bfloat16, (R, self.N)
        px, ldx = _matrix(X, "X", (R, self.K), bf)
        py, ldy = _matrix(Y, "Y", out, bf)
        pr, ldr = (None, 0) if residual is None else _matrix(residual, "residual", out, bf)
        pz, ldz = (None, 0) if Z is None else _matrix(Z, "Z", out, bf)
        _check(self._lib.mlp_linear_forward(
            self._h, R, px, ldx, _dense(W, "W", self.weight_shape, bf),
            None if bias is None else _dense(bias, "bias", self.bias_shape, self.bias_dtype), pr, ldr,
            self._offsets(offsets), pz, ldz, py, ldy, _stream(stream, self.device)), "mlp_linear_forward")

    def backward(self, dY, X, W, *, Z=None, dX=None, dW=None, dbias=None, offsets=None, workspace=None, stream=None):
        """The gradients asked for, of forward() at pre-activation Z (not needed without an activation).  X may be
        None without dW, W without dX.  The residual's gradient is dY itself."""
        R = dY.shape[0]
        bf, inp, out = torch.bfloat16, (R, self.K), (R, self.N)
        act = self.activation != "none"
        pdy, lddy = _matrix(dY, "dY", out, bf)
        px, ldx = _matrix(X, "X", inp, bf) if X is not None or dW is not None else (None, 0)
        pz, ldz = _matrix(Z, "Z", out, bf) if Z is not None or act else (None, 0)
        pdx, lddx = _matrix(dX, "dX", inp, bf) if dX is not None else (None, 0)
        need = self.workspace_size(R) if act or dbias is not None else 0
        _check(self._lib.mlp_linear_backward(
            self._h, R, pdy, lddy, px, ldx,
            _dense(W, "W", self.weight_shape, bf) if W is not None or dX is not None else None, pz, ldz,
            self._offsets(offsets), pdx, lddx, None if dW is None else _dense(dW, "dW", self.weight_shape, self.dw_dtype),
            None if dbias is None else _dense(dbias, "dbias", self.bias_shape, self.bias_dtype),
            _workspace(workspace, need), _stream(stream, self.device)), "mlp_linear_backward")

    def check(self, stream=None) -> int:
        """Synchronise and return the device status (0 = OK); clears it."""
        return int(self._lib.mlp_linear_check(self._h, _stream(stream, self.device)))

    def plan(self, rows: int, what: str = "Y") -> dict:
        """The kernel variant that computes "Y", "dX" or "dW" for this many rows."""
        p = LinearPlan()
        _check(self._lib.mlp_linear_get_plan(self._h, rows, ("Y", "dX", "dW").index(what), ctypes.byref(p)),
               "mlp_linear_get_plan")
        return {"form": ("rows", "rows_t", "reduce")[p.form], "cta_pair": p.cta_pair, "tile_cols": p.tile_cols,
                "k_split": p.k_split, "pipe_stages": p.pipe_stages}

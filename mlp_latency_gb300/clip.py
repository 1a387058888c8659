"""Python binding of include/mlp_clip.h: the norm of all gradients of a step, and clipping by it.

Argument checks and marshalling only, as in block.py.  ``grads`` is a list or tuple of contiguous CUDA tensors of any
shape, bfloat16 or float32, all on norm's device; ``norm`` is float32 [1], ``workspace`` at least
``clip_workspace_size(len(grads))`` bytes.  The workspace lies within no tensor of the lists, nor does the norm when they
are clipped.  A call enqueues work on ``stream`` (default: torch's current stream of that device) without synchronising: a
step that depends on the norm reads it when it likes.
"""
from __future__ import annotations

import ctypes
import functools

from . import _lib
from .chain import MlpChainError, _check

_marshal = None


def _load():
    global _marshal
    _marshal = _lib.load_marshal()
    return _marshal


@functools.lru_cache(maxsize=1024)
def clip_workspace_size(tensors: int) -> int:
    """Bytes of workspace of gradient_norm and clip_gradients for this many tensors."""
    n = ctypes.c_size_t()
    _check(_lib.load().mlp_clip_workspace_size(tensors, ctypes.byref(n)), "mlp_clip_workspace_size")
    return n.value


def gradient_norm(grads, norm, *, workspace=None, stream=None):
    """norm = sqrt(sum of the squares of all elements of all tensors) (mlp_gradient_norm)."""
    status = (_marshal or _load()).clip(grads, None, None, norm, 0.0, workspace, stream)
    if status:
        raise MlpChainError(status, "mlp_gradient_norm")


def clip_gradients(grads, max_norm: float, norm, *, out=None, eps: float = 1e-6, workspace=None, stream=None):
    """norm as gradient_norm's, and every gradient times min(1, max_norm / (norm + eps)), in place or into the tensors of
    ``out`` (mlp_clip_gradients).  In place nothing is written when the factor is 1.  A norm of NaN makes all gradients
    NaN, an infinite gradient makes the finite ones 0."""
    status = (_marshal or _load()).clip(grads, out, float(max_norm), norm, eps, workspace, stream)
    if status:
        raise MlpChainError(status, "mlp_clip_gradients")

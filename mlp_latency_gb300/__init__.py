"""mlp_latency_gb300 -- CTA-pipelined GEMM chains and the operators of an MLP block around them, on one
GB300 (sm_103a).

The compute path is libmlp_chain.so (hand-written tcgen05/TMA CUDA, C ABI in include/mlp_chain.h and
include/mlp_block.h); this package only builds it and marshals arguments to it.
"""
from ._lib import build, load, LIB_PATH  # noqa: F401
from .chain import (Chain, MlpChainError, deps_build, protocol_model, scoreboard_build, EVENT_DTYPE,  # noqa: F401
                    OK, ERR_TIMEOUT, ERR_BAD_TILE, ERR_INVALID_ARG, ERR_UNSUPPORTED)

_BLOCK = ("Linear", "layer_norm_forward", "layer_norm_backward", "layer_norm_workspace_size")


def __getattr__(name):   # the operators take torch tensors: torch is imported with the first use of one
    if name in _BLOCK:
        from . import block
        globals().update({n: getattr(block, n) for n in _BLOCK})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")

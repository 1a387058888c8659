"""GPU tests of layer norm whose weights have another type than the rows, at the widths where the kernels change.

Tolerances: those of test_gpu_layer_norm.py, whose sums and roundings these are.
"""
import numpy as np
import pytest
import torch

import block_reference as ref
from test_gpu_layer_norm import BF, DEV, EPS, F32, close, draw, f64, mc, terms  # noqa: F401

pytestmark = pytest.mark.gpu

# narrow, one and several vectors a thread, the widest rows with gamma in shared memory and without, and rows too wide for registers
SHAPES = [(5, 64), (3, 2048), (320, 520), (320, 4104), (2, 8192), (3, 14336), (3, 14344), (160, 14344), (2, 16384), (2, 25608), (2, 33000),
          (3, 40000)]


def weight(C, seed, dtype, skew, shift=0.0):
    buf = torch.empty(C + skew, dtype=dtype, device=DEV)
    buf[skew:].copy_(draw((C,), seed, dtype, 0.3, shift))
    return buf[skew:]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("wd", [BF, F32])
@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("R,C", SHAPES)
def test_weights_of_either_type(mc, R, C, dtype, wd, skew):  # noqa: F811
    x, dy, r_ = draw((R, C), 1, dtype, 2.0, 0.5), draw((R, C), 4, dtype), draw((R, C), 5, dtype)
    gamma, beta = weight(C, 2, wd, skew, 1.0), weight(C, 3, wd, skew)
    xd, dyd, rd = x.to(DEV), dy.to(DEV), r_.to(DEV)
    y, mean, rstd = torch.full_like(xd, float("nan")), torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    mc.layer_norm_forward(xd, gamma, beta, y, mean=mean, rstd=rstd, eps=EPS)
    want, m, r = ref.norm(f64(x), f64(gamma), f64(beta), EPS)
    n, rnd = terms(C), 2.0 ** -8 if dtype is BF else 0.0
    mag = np.abs(f64(x)).mean(1)
    err = n * 2.0 ** -23 * (np.abs(want) + np.abs(f64(gamma)) * (1 + mag * r)[:, None] + np.abs(f64(beta)))
    close(y, want, err * (1 + np.abs(want)) + rnd * np.abs(want), "y")
    m32, r32 = f64(mean), f64(rstd)
    xh = np.abs((f64(x) - m32[:, None]) * r32[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    scale = r32[:, None] * (g + g.mean(1, keepdims=True) + (xh + 1) * (g * (xh + 1)).mean(1, keepdims=True))
    ws = torch.full((mc.layer_norm_workspace_size(R, C),), 0xff, dtype=torch.uint8, device=DEV)
    for add in (None, rd):
        want, dg, db = ref.norm_grad(f64(dy), f64(x), f64(gamma), m32, r32, None if add is None else f64(r_))
        for sums in (True, False):
            dx = torch.full_like(xd, float("nan"))
            dgamma, dbeta = (torch.full((C,), float("nan"), dtype=wd, device=DEV) for _ in range(2))
            kw = dict(dgamma=dgamma, dbeta=dbeta, workspace=ws) if sums else {}
            mc.layer_norm_backward(dyd, xd, gamma, mean, rstd, dx, dx_add=add, **kw)
            close(dx, want, n * 2.0 ** -23 * (scale + np.abs(want)) + rnd * np.abs(want), f"dx, sums {sums}")
            if sums:
                wr, rel = 2.0 ** -8 if wd is BF else 0.0, (R + 8) * 2.0 ** -24
                close(dgamma, dg, rel * (np.abs(f64(dy)) * (xh + 1)).sum(0) + wr * np.abs(dg), "dgamma")
                close(dbeta, db, rel * np.abs(f64(dy)).sum(0) + wr * np.abs(db), "dbeta")

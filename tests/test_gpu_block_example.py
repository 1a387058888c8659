"""The example's MLP block, dense and with experts, against torch autograd in fp32 on the same bf16 values.

The block rounds h, the activations, dZ and each operator's outputs to bf16 (2^-9 relative each); a gradient passes
through at most eight such roundings, so in norm it is off by 8 * 2^-9 at most; a factor of two for the rest."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
TOL = 2 * 8 * 2.0 ** -9


def reference(block, x, dy):
    p = {k: v.float().clone().requires_grad_() for k, v in block.p.items()}
    xr = x.float().clone().requires_grad_()
    h = torch.nn.functional.layer_norm(xr, (block.width,), p["gamma"], p["beta"])
    mlp = lambda t, e: torch.nn.functional.gelu(t @ p["W1"][e] + p["b1"][e], approximate="tanh") @ p["W2"][e] + p["b2"][e]
    if not block.experts:
        y = xr + mlp(h, ...)
    else:
        gates = torch.softmax(h @ p["Wr"], dim=1)
        chosen = torch.zeros_like(gates).index_put_((block.token, block_expert(block)), torch.ones((), device="cuda"))
        y = xr + sum((gates * chosen)[:, e:e + 1] * mlp(h, e) for e in range(block.experts))
    y.backward(dy.float())
    return y, xr.grad, {k: v.grad for k, v in p.items()}


def block_expert(block):
    """Expert of each routed row, as the block routed it."""
    sizes = (block.offsets[1:] - block.offsets[:-1]).long()
    return torch.repeat_interleave(torch.arange(block.experts, device="cuda"), sizes)


def close(a, b, what):
    err, ref = float((a.float() - b.float()).norm().detach()), float(b.float().norm().detach())
    assert err <= TOL * ref, f"{what}: {err / ref:.4f}"


@pytest.mark.parametrize("experts", [0, 5])
def test_block_matches_autograd(experts):
    import mlp_block
    mlp_block.mc.build()
    torch.manual_seed(3)
    block = mlp_block.MlpBlock(333, 264, 520, experts)
    for k in ("gamma", "beta", "b1", "b2"):
        block.p[k].add_(torch.randn_like(block.p[k]) * 0.3)
    x, dy = torch.randn(333, 264, device="cuda").bfloat16(), torch.randn(333, 264, device="cuda").bfloat16()
    y = block.forward(x)
    dx = block.backward(dy)
    block.check()
    yr, dxr, gr = reference(block, x, dy)
    close(y, yr, "y")
    close(dx, dxr, "dx")
    for k in block.p:
        close(block.grad[k], gr[k], k)

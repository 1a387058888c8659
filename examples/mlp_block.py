"""A pre-norm MLP block, dense or with experts, forward and backward, from the operators of mlp_latency_gb300:

    h = norm(x);   y = x + act(h W1 + b1) W2 + b2                      (dense)
    h = norm(x);   y = x + sum_j g_j (act(h W1[e_j] + b1[e_j]) W2[e_j] + b2[e_j])   (the top experts e_j of a token)

One call per operator; the router of the expert form (a small product, softmax and top-k) is plain torch.

    python examples/mlp_block.py                      # a few SGD steps of each form, loss printed
    python examples/mlp_block.py --rows 4096 --width 8192 --hidden 8192 --steps 20
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mlp_latency_gb300 as mc  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class MlpBlock:
    def __init__(self, rows, width, hidden, experts=0, top=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.width, self.hidden, self.experts, self.top = rows, width, hidden, experts, top if experts else 1
        lead = (experts,) if experts else ()
        n = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(BF)
        self.p = {"gamma": torch.ones(width, dtype=BF, device="cuda"), "beta": torch.zeros(width, dtype=BF, device="cuda"),
                  "W1": n(lead + (width, hidden), width ** -0.5), "b1": torch.zeros(lead + (hidden,), dtype=BF, device="cuda"),
                  "W2": n(lead + (hidden, width), hidden ** -0.5), "b2": torch.zeros(lead + (width,), dtype=BF, device="cuda")}
        if experts:
            self.p["Wr"] = n((width, experts), width ** -0.5)
        self.grad = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.up = mc.Linear(width, hidden, activation="gelu", experts=experts)
        self.down = mc.Linear(hidden, width, experts=experts)
        inner = rows * self.top                        # rows that reach the products
        new = lambda *s, d=BF: torch.empty(*s, dtype=d, device="cuda")
        self.h, self.mean, self.rstd = new(rows, width), new(rows, d=F32), new(rows, d=F32)
        self.z, self.a, self.da = new(inner, hidden), new(inner, hidden), new(inner, hidden)
        self.ws = new(max(self.up.workspace_size(inner), self.down.workspace_size(inner),
                          mc.layer_norm_workspace_size(rows, width)), d=torch.uint8)

    def _route(self):
        """The top experts of every token, the products' rows sorted by expert, and where each expert's begin."""
        self.logits = (self.h.float() @ self.p["Wr"].float()).requires_grad_()
        gates, expert = torch.softmax(self.logits, dim=1).topk(self.top, dim=1)
        expert, order = expert.reshape(-1).sort(stable=True)
        self.token = order // self.top
        self.gates = gates.reshape(-1)[order]
        counts = torch.bincount(expert, minlength=self.experts)
        self.offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)

    def forward(self, x):
        p = self.p
        y = torch.empty_like(x)
        self.x = x
        mc.layer_norm_forward(x, p["gamma"], p["beta"], self.h, mean=self.mean, rstd=self.rstd)
        if not self.experts:
            self.up.forward(self.h, p["W1"], self.a, bias=p["b1"], Z=self.z)
            self.down.forward(self.a, p["W2"], y, bias=p["b2"], residual=x)
            return y
        self._route()
        self.hx = self.h[self.token]
        self.out = torch.empty_like(self.hx)
        self.up.forward(self.hx, p["W1"], self.a, bias=p["b1"], Z=self.z, offsets=self.offsets)
        self.down.forward(self.a, p["W2"], self.out, bias=p["b2"], offsets=self.offsets)
        mixed = torch.zeros(x.shape, dtype=F32, device="cuda").index_add_(0, self.token, self.out.float() * self.gates.detach()[:, None])
        return (x.float() + mixed).to(BF)

    def backward(self, dy):
        """Fills self.grad and returns the gradient of x."""
        p, g = self.p, self.grad
        off = self.offsets if self.experts else None
        rows_in = self.hx if self.experts else self.h
        dout = dy
        if self.experts:
            dout = (dy[self.token].float() * self.gates.detach()[:, None]).to(BF)
        dh = torch.empty_like(rows_in)
        self.down.backward(dout, self.a, p["W2"], dX=self.da, dW=g["W2"], dbias=g["b2"], offsets=off, workspace=self.ws)
        self.up.backward(self.da, rows_in, p["W1"], Z=self.z, dX=dh, dW=g["W1"], dbias=g["b1"], offsets=off, workspace=self.ws)
        if self.experts:   # back to tokens, with the router's part
            self.gates.backward((dy[self.token].float() * self.out.float()).sum(1))
            dl = self.logits.grad
            g["Wr"].copy_(self.h.float().t() @ dl)
            dh = (torch.zeros(self.h.shape, dtype=F32, device="cuda").index_add_(0, self.token, dh.float())
                  + dl @ p["Wr"].float().t()).to(BF)
        dx = torch.empty_like(self.x)
        mc.layer_norm_backward(dh, self.x, p["gamma"], self.mean, self.rstd, dx, dgamma=g["gamma"], dbeta=g["beta"], dx_add=dy,
                               workspace=self.ws)
        return dx

    def check(self):
        if self.up.check() or self.down.check():
            raise RuntimeError("a product reported a device error")


def train(block, steps, rate):
    """Regress the block's output on a fixed target; returns the losses."""
    x = torch.randn(block.rows, block.width, device="cuda").to(BF)
    target = torch.randn(block.rows, block.width, device="cuda").to(BF)
    losses = []
    for _ in range(steps):
        diff = block.forward(x).float() - target.float()
        losses.append(float(diff.square().mean()))
        block.backward((diff * (2.0 / diff.numel())).to(BF))
        for k, v in block.p.items():
            v.add_(block.grad[k], alpha=-rate)
    block.check()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--rate", type=float, default=5.0)
    a = ap.parse_args()
    mc.build()
    torch.manual_seed(0)
    for name, experts in (("dense", 0), (f"{a.experts} experts", a.experts)):
        losses = train(MlpBlock(a.rows, a.width, a.hidden, experts), a.steps, a.rate)
        print(f"{name}: loss {losses[0]:.4f} -> {losses[-1]:.4f} over {a.steps} steps")

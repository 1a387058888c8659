"""GPU tests of mlp_linear calls among other calls."""
import pytest
import torch

import seeded_inputs as si
from test_gpu_linear import BF, DEV, mc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["pipelined", "sequential"])
def test_an_error_is_not_left_for_a_later_call(mc, mode):  # noqa: F811
    w = si.WORKLOADS["tiny_m64_d256"]
    X, Ws = si.draw(w, seed=0)
    X, Ws = X.to(DEV), [t.to(DEV) for t in Ws]
    with mc.Chain(w.M, w.dims, tile_n=[64, 64], mode=mode) as ch:
        ws = torch.empty(max(ch.workspace_size(), 256), dtype=torch.uint8, device=DEV)
        Y = [torch.full((w.M, w.dims[-1]), float("nan"), dtype=BF, device=DEV) for _ in range(2)]
        ch.run(X, Ws, Y[0], ws)
        with pytest.raises(mc.MlpChainError):
            mc.Linear(64, 64, device=99)
        ch.run(X, Ws, Y[1], ws)
        assert ch.check() == 0
    assert torch.equal(Y[0], Y[1])


def test_tensors_of_another_device_are_refused(mc):  # noqa: F811
    """The checks of a handle on cuda:1, which need no such device: no handle is behind them, and every tensor is on cuda:0."""
    from mlp_latency_gb300 import _lib
    K, N, rows = 64, 72, 10
    t = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
    marshal = _lib.load_marshal()
    X, W, Y, ws = t(rows, K), t(K, N), t(rows, N), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for device, says in ((1, "on cuda:1, got"), (0, None)):
        args = marshal.linear(0, K, N, 0, 0, 0, 1, 1, device)
        calls = [lambda: marshal.linear_forward(args, X, W, Y, None, None, None, None, 0),
                 lambda: marshal.linear_backward(args, Y, None, None, None, None, None, None, None, None, 0)]
        for call in calls:
            if says:
                with pytest.raises(ValueError, match=says):
                    call()
            else:
                assert call() == mc.ERR_INVALID_ARG
    with mc.Linear(K, N, activation="gelu") as lin:
        f = dict(bias=t(N), residual=Y, Z=t(rows, N))
        for name in ("X", "W", "Y", *f):
            a = dict(X=X, W=W, Y=t(rows, N), **f)
            a[name] = a[name].cpu()
            with pytest.raises(ValueError, match=f"{name}: expected a .*CUDA tensor"):
                lin.forward(a.pop("X"), a.pop("W"), a.pop("Y"), **a)
        b = dict(Z=t(rows, N), dX=t(rows, K), dW=t(K, N), dbias=t(N), workspace=ws)
        for name in ("dY", "X", "W", *b):
            a = dict(dY=Y, X=X, W=W, **b)
            a[name] = a[name].cpu()
            with pytest.raises(ValueError, match=f"{name}: expected a .*CUDA tensor"):
                lin.backward(a.pop("dY"), a.pop("X"), a.pop("W"), **a)


def test_layer_norm_arguments_of_another_device_are_refused(mc):  # noqa: F811
    R, C = 4, 64
    t = lambda *s: torch.ones(*s, device=DEV)  # noqa: E731
    f = dict(x=t(R, C), gamma=t(C), beta=t(C), y=t(R, C), mean=t(R), rstd=t(R))
    b = dict(dy=t(R, C), x=t(R, C), gamma=t(C), mean=t(R), rstd=t(R), dx=t(R, C), dgamma=t(C), dbeta=t(C), dx_add=t(R, C),
             workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    for call, good in ((mc.layer_norm_forward, f), (mc.layer_norm_backward, b)):
        call(**good)
        for name in good:
            a = dict(good)
            a[name] = a[name].cpu()
            with pytest.raises(ValueError, match=": expected a .*CUDA tensor"):
                call(**a)


def test_a_handle_does_not_grow_with_its_calls(mc):  # noqa: F811
    """A served batch has another number of rows from call to call."""
    import sys
    with mc.Linear(64, 64, activation="gelu") as lin:
        def size():
            return sum(sys.getsizeof(v) for v in vars(lin).values())
        lin.workspace_size(1)
        before = size()
        for rows in range(1, 3000):
            assert lin.workspace_size(rows) >= rows * 64 * 2
        assert size() == before

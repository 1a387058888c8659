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

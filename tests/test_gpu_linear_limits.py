"""GPU tests of mlp_linear at the ends of what it accepts, and past them: bad offsets."""
import pytest
import torch

from test_gpu_linear import BF, DEV, blank, draw, mc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets", [[0, 120, 90], [0, 60, 120], [-4, 60, 100], [70, 60, 100]])
@pytest.mark.parametrize("what", ["dbias", "dX", "dW", "all"])
def test_bad_offsets_of_a_gradient_are_reported(mc, offsets, what):  # noqa: F811
    rows, K, N = 100, 64, 72
    X, W, dY = draw((rows, K), 1.0, 1).to(DEV), draw((2, K, N), 0.1, 2).to(DEV), draw((rows, N), 1.0, 3).to(DEV)
    out = {"dX": blank(rows, K, 0), "dW": torch.empty_like(W), "dbias": torch.empty(2, N, dtype=BF, device=DEV)}
    asked = out if what == "all" else {what: out[what]}
    with mc.Linear(K, N, experts=2) as lin:
        ws = torch.empty(lin.workspace_size(rows), dtype=torch.uint8, device=DEV)
        for off, status in ((offsets, mc.ERR_INVALID_ARG), ([0, 60, 100], 0)):
            lin.backward(dY, X, W, offsets=torch.tensor(off, dtype=torch.int32, device=DEV), workspace=ws, **asked)
            assert lin.check() == status


def test_a_reduction_over_very_many_rows_is_within_the_default_limit(mc):  # noqa: F811
    """600 million rows, of which only the last are not zero: exact."""
    rows, n, last = 600_000_000, 8, 5
    X, dY = (torch.zeros(rows, n, dtype=BF, device=DEV) for _ in range(2))
    X[-last:] = torch.arange(last * n, device=DEV).view(last, n).to(BF)
    dY[-last:] = torch.arange(last * n, device=DEV).view(last, n).flip(0).to(BF)
    dW = torch.full((n, n), float("nan"), device=DEV)
    with mc.Linear(n, n, dw_dtype=torch.float32) as lin:
        lin.backward(dY, X, None, dW=dW)
        assert lin.check() == 0
    assert torch.equal(dW.cpu().double(), X[-last:].cpu().double().t() @ dY[-last:].cpu().double())

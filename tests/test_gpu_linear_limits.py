"""GPU tests of mlp_linear at the ends of what it accepts."""
import pytest
import torch

from test_gpu_linear import BF, DEV, F32, mc  # noqa: F401

pytestmark = pytest.mark.gpu
MOST_ROWS = 2 ** 31 - 1024


def test_bias_gradient_of_the_most_rows(mc):  # noqa: F811
    """The last rows count too: all others are zero, so the sums are exact."""
    N = 8
    dY = torch.zeros(MOST_ROWS, N, dtype=BF, device=DEV)
    dY[-3:] = torch.arange(1, 1 + 3 * N, device=DEV).view(3, N).to(BF)
    db = torch.full((N,), float("nan"), device=DEV)
    with mc.Linear(8, N, bias_dtype=F32) as lin:
        ws = torch.full((lin.workspace_size(MOST_ROWS),), 0xff, dtype=torch.uint8, device=DEV)
        lin.backward(dY, None, None, dbias=db, workspace=ws)
        assert lin.check() == 0
    assert torch.equal(db, dY[-3:].float().sum(0))

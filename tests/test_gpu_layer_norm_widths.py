"""GPU tests of layer norm rows as wide as the entries accept.  Sums are of whole
numbers, or of terms whose loss would not show; results are rounded to bf16."""
import pytest
import torch

from test_gpu_layer_norm import BF, DEV, mc  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("C", [2 ** 30 - 1, 2 ** 30 + 1, MOST - 7, MOST])
def test_dx_alone_of_the_widest_rows(mc, C):  # noqa: F811
    """With mean 0, rstd 1 and x = 0: dx = dy - mean(dy), where dy is 1 in the last columns."""
    n = 4096
    x, dy = torch.zeros(1, C, dtype=BF, device=DEV), torch.zeros(1, C, dtype=BF, device=DEV)
    dy[0, -n:] = 1.0
    dx = torch.full((1, C), float("nan"), dtype=BF, device=DEV)
    mc.layer_norm_backward(dy, x, None, torch.zeros(1, device=DEV), torch.ones(1, device=DEV), dx)
    assert bool((dx[0, -n:] == 1.0).all())
    rest = dx[0, :-n]
    assert float(rest.min()) >= -n / C * (1 + 2.0 ** -8) and float(rest.max()) <= -n / C * (1 - 2.0 ** -8)


@pytest.mark.parametrize("C", [MOST - 7, MOST])
def test_forward_of_the_widest_rows(mc, C):  # noqa: F811
    """x is 1 in the last columns: mean m = n / C and variance m (1 - m), of which the other columns' share is m = 2e-6."""
    n = 4096
    x = torch.zeros(1, C, dtype=BF, device=DEV)
    x[0, -n:] = 1.0
    y = torch.full((1, C), float("nan"), dtype=BF, device=DEV)
    mean, rstd = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    mc.layer_norm_forward(x, None, None, y, mean=mean, rstd=rstd, eps=0.0)
    m = n / C
    r = (m * (1 - m)) ** -0.5
    assert abs(float(mean) - m) <= 2.0 ** -23 * m and abs(float(rstd) - r) <= 1e-5 * r
    tol = 1e-5 + 2.0 ** -8
    ones, rest = y[0, -n:], y[0, :-n]
    for t, want in ((ones, (1 - m) * r), (rest, -m * r)):
        assert abs(float(t.min()) - want) <= tol * abs(want) and abs(float(t.max()) - want) <= tol * abs(want)

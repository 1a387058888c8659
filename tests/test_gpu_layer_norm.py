"""GPU tests of layer norm, forward and backward, against 64-bit definitions.

Tolerances.  Sums over C columns are taken in fp32 as per-thread sums of at most 64 terms (1024 where a row does
not fit registers) followed by trees: relative error of a mean of magnitudes below n 2^-24 with n = 80 (1100).
xh then is off by n 2^-23 (|xh| + |mean| rstd): the second term is the rounding of the mean itself.  Results
rounded to bf16 add 2^-8 of themselves.  Column sums over R rows: R 2^-24 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def mc():
    import mlp_latency_gb300
    mlp_latency_gb300.build()
    mlp_latency_gb300.load()
    return mlp_latency_gb300


def draw(shape, seed, dtype, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def place(t, extra, skew):
    """On the device, rows `extra` elements further apart, starting `skew` elements into the buffer."""
    R, C = t.shape
    buf = torch.full((R * (C + extra) + skew,), float("nan"), dtype=t.dtype, device=DEV)
    v = buf[skew:].view(R, C + extra)[:, :C]
    v.copy_(t)
    return v


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(got, want, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.abs(got - want)[bad].max()}"


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 8), (2, 31), (4, 64), (7, 255), (9, 256), (3, 1000), (2, 1025), (6, 1357), (5, 2048), (3, 4099),
          (300, 520), (2, 8192), (1, 8200), (2, 12001), (1, 16384), (1, 33000), (1, 70001)]
LAYOUTS = [(0, 0), (8, 0), (2, 0), (1, 1)]


def terms(C):
    return 80 if C <= 4096 else 1100


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("extra,skew", LAYOUTS)
def test_forward(mc, shape, dtype, extra, skew):
    R, C = shape
    x = draw(shape, 1, dtype, 2.0, 0.5)
    wd = F32 if (C + extra) % 2 else BF
    gamma, beta = draw((C,), 2, wd, 0.3, 1.0), draw((C,), 3, wd, 0.3)
    y = place(torch.full(shape, float("nan"), dtype=dtype), extra, skew)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    mc.layer_norm_forward(place(x, extra, skew), gamma.to(DEV), beta.to(DEV), y, mean=mean, rstd=rstd, eps=EPS)
    want, m, r = ref.norm(f64(x), f64(gamma), f64(beta), EPS)
    n = terms(C)
    mag = np.abs(f64(x)).mean(1)
    close(mean, m, n * 2.0 ** -24 * mag + 1e-30, "mean")
    close(rstd, r, n * 2.0 ** -23 * r * (1 + mag * r), "rstd")
    err = n * 2.0 ** -23 * (np.abs(want) + np.abs(f64(gamma)) * (1 + mag * r)[:, None] + np.abs(f64(beta)))
    close(y, want, err * (1 + np.abs(want)) + (2.0 ** -8 * np.abs(want) if dtype is BF else 0), "y")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("extra,skew", LAYOUTS)
@pytest.mark.parametrize("add", [False, True])
def test_backward(mc, shape, dtype, extra, skew, add):
    R, C = shape
    x, dy, r_ = draw(shape, 1, dtype, 2.0, 0.5), draw(shape, 4, dtype), draw(shape, 5, dtype)
    wd = F32 if (C + extra) % 2 else BF
    gamma = draw((C,), 2, wd, 0.3, 1.0)
    _, m, r = ref.norm(f64(x), None, None, EPS)
    mean, rstd = torch.from_numpy(m).float().to(DEV), torch.from_numpy(r).float().to(DEV)
    dx = place(torch.full(shape, float("nan"), dtype=dtype), extra, skew)
    dgamma, dbeta = torch.full((C,), float("nan"), dtype=wd, device=DEV), torch.full((C,), float("nan"), dtype=wd, device=DEV)
    ws = torch.full((mc.layer_norm_workspace_size(R, C),), 0xff, dtype=torch.uint8, device=DEV)
    mc.layer_norm_backward(place(dy, extra, skew), place(x, extra, skew), gamma.to(DEV), mean, rstd, dx, dgamma=dgamma,
                           dbeta=dbeta, dx_add=place(r_, extra, skew) if add else None, workspace=ws)
    m32, r32 = f64(mean), f64(rstd)
    want, dg, db = ref.norm_grad(f64(dy), f64(x), f64(gamma), m32, r32, f64(r_) if add else None)
    xh = np.abs((f64(x) - m32[:, None]) * r32[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    n = terms(C)
    scale = r32[:, None] * (g + g.mean(1, keepdims=True) + (xh + 1) * (g * (xh + 1)).mean(1, keepdims=True))
    close(dx, want, n * 2.0 ** -23 * (scale + np.abs(want)) + (2.0 ** -8 * np.abs(want) if dtype is BF else 0), "dx")
    rnd = 2.0 ** -8 if wd is BF else 0.0
    rel = (R + 8) * 2.0 ** -24
    close(dgamma, dg, rel * (np.abs(f64(dy)) * (xh + 1)).sum(0) + rnd * np.abs(dg), "dgamma")
    close(dbeta, db, rel * np.abs(f64(dy)).sum(0) + rnd * np.abs(db), "dbeta")


@pytest.mark.parametrize("R,C", [(1000, 264), (2000, 1000), (3000, 4096), (700, 8192), (129, 1357)])
def test_backward_many_rows_repeats_its_bits(mc, R, C):
    x, dy = draw((R, C), 1, BF), draw((R, C), 2, BF)
    gamma = draw((C,), 3, F32, 0.3, 1.0)
    _, m, r = ref.norm(f64(x), None, None, EPS)
    mean, rstd = torch.from_numpy(m).float().to(DEV), torch.from_numpy(r).float().to(DEV)
    ws = torch.empty(mc.layer_norm_workspace_size(R, C), dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(3):
        dx, dg, db = torch.empty(R, C, dtype=BF, device=DEV), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        mc.layer_norm_backward(dy.to(DEV), x.to(DEV), gamma.to(DEV), mean, rstd, dx, dgamma=dg, dbeta=db, workspace=ws)
        outs.append((dx, dg, db))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))
    want, dg, db = ref.norm_grad(f64(dy), f64(x), f64(gamma), f64(mean), f64(rstd), None)
    xh = np.abs((f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    scale = f64(rstd)[:, None] * (g + g.mean(1, keepdims=True) + (xh + 1) * (g * (xh + 1)).mean(1, keepdims=True))
    close(outs[0][0], want, terms(C) * 2.0 ** -23 * (scale + np.abs(want)) + 2.0 ** -8 * np.abs(want), "dx")
    close(outs[0][1], dg, (R + 8) * 2.0 ** -24 * (np.abs(f64(dy)) * (xh + 1)).sum(0), "dgamma")
    close(outs[0][2], db, (R + 8) * 2.0 ** -24 * np.abs(f64(dy)).sum(0), "dbeta")


def test_large_mean_does_not_cancel(mc):
    """Deviations of 1 around 1000: a difference of raw moments would lose them in fp32."""
    x = draw((4, 4096), 9, F32, 1.0, 1000.0)
    y, rstd = torch.empty(4, 4096, device=DEV), torch.empty(4, device=DEV)
    mc.layer_norm_forward(x.to(DEV), None, None, y, rstd=rstd, eps=0.0)
    want, m, r = ref.norm(f64(x), None, None, 0.0)
    # the fp32 mean is off by 80 2^-24 of 1000 (5e-3 of a deviation); its square enters the variance
    close(rstd, r, 5e-5 * r, "rstd")
    close(y, want, 80 * 2.0 ** -24 * 1000 * r[:, None] + 1e-4 * np.abs(want), "y")


def test_constant_and_non_finite_rows(mc):
    x = torch.zeros(4, 264, device=DEV)
    x[0] = 3.0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = torch.arange(264, device=DEV)
    y = torch.empty_like(x)
    mc.layer_norm_forward(x, None, None, y, eps=EPS)
    assert not bool(y[0].any())
    assert bool(torch.isnan(y[1]).any()) and bool(torch.isnan(y[2]).all())
    want, _, _ = ref.norm(f64(x[3:4]), None, None, EPS)
    close(y[3:4], want, 1e-5 * (1 + np.abs(want)), "y")


def test_in_place_and_optional_outputs(mc):
    R, C = 33, 520
    x, dy, add = draw((R, C), 1, BF).to(DEV), draw((R, C), 2, BF).to(DEV), draw((R, C), 3, BF).to(DEV)
    gamma = draw((C,), 4, BF, 0.3, 1.0).to(DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    mc.layer_norm_forward(x, gamma, None, y, mean=mean, rstd=rstd)
    x2 = x.clone()
    mc.layer_norm_forward(x2, gamma, None, x2)
    assert torch.equal(x2, y)
    ws = torch.empty(mc.layer_norm_workspace_size(R, C), dtype=torch.uint8, device=DEV)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    mc.layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db, dx_add=add, workspace=ws)
    for which in ("dy", "x", "add"):
        t = {"dy": dy.clone(), "x": x.clone(), "add": add.clone()}
        dg2, db2 = torch.empty_like(gamma), torch.empty_like(gamma)
        mc.layer_norm_backward(t["dy"], t["x"], gamma, mean, rstd, t[which], dgamma=dg2, dbeta=db2, dx_add=t["add"],
                               workspace=ws)
        assert torch.equal(t[which], dx) and torch.equal(dg, dg2) and torch.equal(db, db2), which
    dx2, dg2, db2 = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    mc.layer_norm_backward(dy, x, gamma, mean, rstd, dx2, dx_add=add)
    mc.layer_norm_backward(dy, x, gamma, mean, rstd, None, dgamma=dg2, workspace=ws)
    mc.layer_norm_backward(dy, x, gamma, mean, rstd, None, dbeta=db2, workspace=ws)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_gradient_against_differences(mc):
    R, C = 6, 72
    x, gamma, beta, G = draw((R, C), 1, F32, 2.0), draw((C,), 2, F32, 0.3, 1.0), draw((C,), 3, F32), draw((R, C), 4, F32)
    mean, rstd, y = torch.empty(R, device=DEV), torch.empty(R, device=DEV), torch.empty(R, C, device=DEV)
    dx, dg, db = torch.empty(R, C, device=DEV), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    ws = torch.empty(mc.layer_norm_workspace_size(R, C), dtype=torch.uint8, device=DEV)
    mc.layer_norm_forward(x.to(DEV), gamma.to(DEV), beta.to(DEV), y, mean=mean, rstd=rstd, eps=EPS)
    mc.layer_norm_backward(G.to(DEV), x.to(DEV), gamma.to(DEV), mean, rstd, dx, dgamma=dg, dbeta=db, workspace=ws)
    base = [f64(x), f64(gamma), f64(beta)]
    rng = np.random.default_rng(3)
    h = 1e-6
    for i, got in enumerate((dx, dg, db)):
        U = rng.standard_normal(base[i].shape)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * U, base[i] - h * U
        num = ((ref.norm(*up, EPS)[0] - ref.norm(*dn, EPS)[0]) * f64(G)).sum() / (2 * h)
        scale = np.abs(f64(got) * U).sum()
        assert abs((f64(got) * U).sum() - num) <= 2.0 ** -14 * scale


def test_zero_rows(mc):
    e = torch.empty(0, 64, device=DEV)
    g = torch.ones(64, device=DEV)
    n = torch.empty(0, device=DEV)
    mc.layer_norm_forward(e, g, g, e)
    dg, db = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    ws = torch.empty(max(mc.layer_norm_workspace_size(0, 64), 256), dtype=torch.uint8, device=DEV)
    mc.layer_norm_backward(e, e, g, n, n, e, dgamma=dg, dbeta=db, workspace=ws)
    assert not bool(dg.any()) and not bool(db.any())


def test_refusals_of_tensors(mc):
    t = lambda *s, d=F32: torch.empty(*s, dtype=d, device=DEV)
    x, g, y = t(4, 64), t(64), t(4, 64)
    for a in ((x.half(), g, g, y), (x, t(65), g, y), (x, g, g.to(BF), y), (x, g, g, t(4, 65)), (x, g, g, t(4, 64, d=BF)), (x, g, g, None),
              (t(64, 4).t(), g, g, y), (t(64), g, g, y)):
        with pytest.raises(ValueError):
            mc.layer_norm_forward(*a)
    with pytest.raises(ValueError):
        mc.layer_norm_forward(x, g, g, y, mean=t(5))
    with pytest.raises(mc.MlpChainError):
        mc.layer_norm_forward(x, g, g, y, eps=-1.0)
    with pytest.raises(mc.MlpChainError):      # dgamma without a workspace
        mc.layer_norm_backward(x, x, g, t(4), t(4), y, dgamma=g)
    with pytest.raises(ValueError):
        mc.layer_norm_backward(x, x, g, t(4), t(4), y, dgamma=g, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        mc.layer_norm_backward(x, x, g, None, t(4), y)


ODD_ROWS = [(700, 300, 300), (1400, 1357, 1357), (400, 5111, 5120), (400, 5111, 5111), (333, 8189, 8195), (310, 11249, 11249),
            (310, 12001, 12003), (17, 16383, 16383), (9, 16378, 16378), (2, 517, 523)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C,ld", ODD_ROWS)
@pytest.mark.parametrize("add", [False, True])
def test_rows_that_start_inside_a_word(mc, R, C, ld, dtype, add):
    """Many rows whose ends lie inside 16-byte words.  NaN between the rows is neither used nor overwritten, and neither is
    the row before or after."""
    x, dy, r_ = draw((R, C), 1, dtype, 2.0, 0.5), draw((R, C), 4, dtype), draw((R, C), 5, dtype)
    gamma, beta = draw((C,), 2, F32, 0.3, 1.0), draw((C,), 3, F32, 0.3)
    nan = torch.full((R, C), float("nan"), dtype=dtype)
    xd, dyd = place(x, ld - C, 0), place(dy, ld - C, 0)
    y, dx = place(nan, ld - C, 0), place(nan, ld - C, 0)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    mc.layer_norm_forward(xd, gamma.to(DEV), beta.to(DEV), y, mean=mean, rstd=rstd, eps=EPS)
    want, m, r = ref.norm(f64(x), f64(gamma), f64(beta), EPS)
    n, rnd = terms(C), 2.0 ** -8 if dtype is BF else 0.0
    mag = np.abs(f64(x)).mean(1)
    close(mean, m, n * 2.0 ** -24 * mag + 1e-30, "mean")
    close(rstd, r, n * 2.0 ** -23 * r * (1 + mag * r), "rstd")
    err = n * 2.0 ** -23 * (np.abs(want) + np.abs(f64(gamma)) * (1 + mag * r)[:, None] + np.abs(f64(beta)))
    close(y, want, err * (1 + np.abs(want)) + rnd * np.abs(want), "y")
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    ws = torch.full((mc.layer_norm_workspace_size(R, C),), 0xff, dtype=torch.uint8, device=DEV)
    mc.layer_norm_backward(dyd, xd, gamma.to(DEV), mean, rstd, dx, dgamma=dg, dbeta=db,
                           dx_add=place(r_, ld - C, 0) if add else None, workspace=ws)
    m32, r32 = f64(mean), f64(rstd)
    want, wg, wb = ref.norm_grad(f64(dy), f64(x), f64(gamma), m32, r32, f64(r_) if add else None)
    xh = np.abs((f64(x) - m32[:, None]) * r32[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    scale = r32[:, None] * (g + g.mean(1, keepdims=True) + (xh + 1) * (g * (xh + 1)).mean(1, keepdims=True))
    close(dx, want, n * 2.0 ** -23 * (scale + np.abs(want)) + rnd * np.abs(want), "dx")
    rel = (R + 8) * 2.0 ** -24
    close(dg, wg, rel * (np.abs(f64(dy)) * (xh + 1)).sum(0), "dgamma")
    close(db, wb, rel * np.abs(f64(dy)).sum(0), "dbeta")
    for out in (y, dx):
        gaps = torch.as_strided(out, (R, ld - C), (ld, 1), C)
        assert torch.isnan(gaps).all()


@pytest.mark.parametrize("R,C", [(700, 1357), (400, 5111), (310, 11249)])
def test_in_place_rows_that_start_inside_a_word(mc, R, C):
    """dx over dy, and y over x, where a word holds the end of one row and the start of the next: the same bits as elsewhere."""
    x, dy = draw((R, C), 1, BF, 2.0, 0.5).to(DEV), draw((R, C), 4, BF).to(DEV)
    gamma, beta = draw((C,), 2, F32, 0.3, 1.0).to(DEV), draw((C,), 3, F32, 0.3).to(DEV)
    mean, rstd, y, dx = torch.empty(R, device=DEV), torch.empty(R, device=DEV), torch.empty_like(x), torch.empty_like(x)
    mc.layer_norm_forward(x, gamma, beta, y, mean=mean, rstd=rstd, eps=EPS)
    mc.layer_norm_backward(dy, x, gamma, mean, rstd, dx)
    over = dy.clone()
    mc.layer_norm_backward(over, x, gamma, mean, rstd, over)
    assert torch.equal(over, dx)
    over = x.clone()
    mc.layer_norm_forward(over, gamma, beta, over, eps=EPS)
    assert torch.equal(over, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C", [(5, 300), (400, 1357), (320, 5111), (3, 16379)])
def test_arrays_whose_rows_start_at_different_places(mc, R, C, dtype):
    """The same results, up to rounding, as for arrays of equal strides."""
    x, dy, r_ = draw((R, C), 1, dtype, 2.0, 0.5), draw((R, C), 4, dtype), draw((R, C), 5, dtype)
    gamma, beta = draw((C,), 2, BF, 0.3, 1.0), draw((C,), 3, BF, 0.3)
    nan = torch.full((R, C), float("nan"), dtype=dtype)
    y, dx = place(nan, 3, 0), place(nan, 2, 1)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    mc.layer_norm_forward(place(x, 0, 0), gamma.to(DEV), beta.to(DEV), y, mean=mean, rstd=rstd, eps=EPS)
    want, m, r = ref.norm(f64(x), f64(gamma), f64(beta), EPS)
    n, rnd = terms(C), 2.0 ** -8 if dtype is BF else 0.0
    mag = np.abs(f64(x)).mean(1)
    err = n * 2.0 ** -23 * (np.abs(want) + np.abs(f64(gamma)) * (1 + mag * r)[:, None] + np.abs(f64(beta)))
    close(y, want, err * (1 + np.abs(want)) + rnd * np.abs(want), "y")
    dg, db = torch.empty(C, dtype=BF, device=DEV), torch.empty(C, dtype=BF, device=DEV)
    ws = torch.full((mc.layer_norm_workspace_size(R, C),), 0xff, dtype=torch.uint8, device=DEV)
    mc.layer_norm_backward(place(dy, 1, 0), place(x, 0, 0), gamma.to(DEV), mean, rstd, dx, dgamma=dg, dbeta=db,
                           dx_add=place(r_, 5, 0), workspace=ws)
    m32, r32 = f64(mean), f64(rstd)
    want, wg, wb = ref.norm_grad(f64(dy), f64(x), f64(gamma), m32, r32, f64(r_))
    xh = np.abs((f64(x) - m32[:, None]) * r32[:, None])
    g = np.abs(f64(dy) * f64(gamma))
    scale = r32[:, None] * (g + g.mean(1, keepdims=True) + (xh + 1) * (g * (xh + 1)).mean(1, keepdims=True))
    close(dx, want, n * 2.0 ** -23 * (scale + np.abs(want)) + rnd * np.abs(want), "dx")
    rel = (R + 8) * 2.0 ** -24
    close(dg, wg, rel * (np.abs(f64(dy)) * (xh + 1)).sum(0) + 2.0 ** -8 * np.abs(wg), "dgamma")
    close(db, wb, rel * np.abs(f64(dy)).sum(0) + 2.0 ** -8 * np.abs(wb), "dbeta")

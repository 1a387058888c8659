"""GPU tests of mlp_linear: forward and backward, dense and by expert, against 64-bit products.

Tolerances.  Products of bf16 numbers are exact in fp32; the tensor cores add 16 of them at a time to an fp32
accumulator, each addition off by at most 2^-22 of the sum of absolute terms S (truncation included), K/16 + 1
additions plus at most 8 partial sums, the bias and the residual: E = (K/16 + 16) 2^-22 S.  Activations have
slope below 1.2 and are evaluated to 2^-18 of |z| + 1.  A bf16 result adds half a unit, 2^-8 |y| at most.  In the
backward pass dZ is rounded to bf16 before the products: another 2^-8 S.
"""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mc():
    import mlp_latency_gb300
    mlp_latency_gb300.build()
    mlp_latency_gb300.load()
    return mlp_latency_gb300


def draw(shape, std, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def wide(t, extra):
    """The same values as a slice of a wider matrix."""
    if not extra:
        return t.to(DEV)
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    w[:, 8:8 + t.shape[1]] = t.to(DEV)
    return w[:, 8:8 + t.shape[1]]


def blank(rows, cols, extra, dtype=BF):
    return torch.full((rows, cols + extra), float("nan"), dtype=dtype, device=DEV)[:, :cols]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def check_close(got, want, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.abs(got - want)[bad].max()}"


def run_forward(mc, rows, K, N, act, layout, counts=None, first=0, bias="bf16", residual=True, save=True, extra=0,
                seed=0):
    E = len(counts) if counts is not None else 0
    lead = (E,) if E else ()
    X = draw((rows, K), 1.0, seed)
    W = draw(lead + ((K, N) if layout == "kn" else (N, K)), K ** -0.5, seed + 1)
    b = draw(lead + (N,), 0.5, seed + 2, BF if bias == "bf16" else F32) if bias else None
    R = draw((rows, N), 1.0, seed + 3) if residual else None
    off = offsets_of(counts, first) if E else None
    Y = blank(rows, N, extra)
    Z = blank(rows, N, extra) if save else None
    with mc.Linear(K, N, activation=act, experts=E, weight_layout=layout,
                   bias_dtype=F32 if bias == "f32" else BF) as lin:
        lin.forward(wide(X, extra), W.to(DEV), Y, bias=b.to(DEV) if bias else None,
                    residual=wide(R, extra) if residual else None, Z=Z,
                    offsets=torch.from_numpy(off).to(DEV) if E else None)
        assert lin.check() == 0
    y, z, S = ref.linear(f64(X), f64(W), f64(b), f64(R), act, layout, off)
    used = ~np.isnan(S[:, 0])
    E_acc = (K / 16 + 16) * 2.0 ** -22 * S[used]
    if save:
        check_close(Z[torch.from_numpy(used)], z[used], E_acc + 2.0 ** -8 * np.abs(z[used]), "Z")
        assert bool(torch.isnan(Z[torch.from_numpy(~used)].float()).all())
    tol = 1.2 * E_acc + 2.0 ** -18 * (np.abs(z[used]) + 1) + 2.0 ** -8 * np.abs(y[used])
    check_close(Y[torch.from_numpy(used)], y[used], tol, "Y")
    assert bool(torch.isnan(Y[torch.from_numpy(~used)].float()).all())
    if extra:   # nothing is stored beside the slice
        assert bool(torch.isnan(Y.as_strided((rows, extra), (N + extra, 1), N).float()).all())


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("rows,K,N", [(1, 8, 8), (1, 4096, 520), (2, 72, 264), (31, 200, 1000), (33, 1000, 200), (64, 64, 136),
                                      (65, 520, 256), (127, 128, 40), (129, 264, 1032), (257, 72, 520), (300, 2048, 264),
                                      (513, 136, 2056)])
def test_forward_odd_sizes(mc, rows, K, N, layout):
    run_forward(mc, rows, K, N, "gelu", layout, seed=rows + K)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("bias,residual,save", [(None, False, False), ("f32", False, True), ("bf16", True, False)])
def test_forward_epilogues(mc, act, rows, bias, residual, save):
    run_forward(mc, rows, 264, 328, act, "kn", bias=bias, residual=residual, save=save, seed=7)


@pytest.mark.parametrize("rows,extra", [(3, 24), (40, 8), (150, 16), (700, 24)])
def test_forward_strided(mc, rows, extra):
    run_forward(mc, rows, 328, 520, "silu", "nk", extra=extra, seed=11)


def test_forward_every_variant(mc):
    """One run for each kernel variant (form, pair, tile, split) that the rule picks over a grid of sizes."""
    seen = {}
    for K in (64, 512, 4096, 8192):
        for N in (256, 512, 1024, 2048, 8192, 20480):
            with mc.Linear(K, N) as lin:
                for rows in (4, 24, 60, 100, 130, 250, 500, 2048):
                    p = lin.plan(rows)
                    key = (p["form"], p["cta_pair"], p["tile_cols"], p["k_split"])
                    if key not in seen or rows * K * N < np.prod(seen[key]):
                        seen[key] = (rows, K, N)
    assert {"rows", "rows_t"} <= {k[0] for k in seen} and {1, 2} <= {k[1] for k in seen}
    assert any(k[0] == "rows" and k[3] > 1 for k in seen) and any(k[0] == "rows_t" and k[3] > 1 for k in seen)
    for i, (rows, K, N) in enumerate(seen.values()):
        run_forward(mc, rows, K, N, "gelu", "nk" if i % 2 else "kn", seed=13)


COUNTS = [[0, 0, 0], [1], [0, 5, 0, 0, 1, 30, 0], [64, 0, 128, 1, 63], [300, 0, 17, 256, 129], [3] * 70,
          [700, 1, 0, 0, 299]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("layout,act", [("kn", "silu"), ("nk", "gelu")])
def test_forward_experts(mc, counts, layout, act):
    run_forward(mc, max(sum(counts), 1), 264, 392, act, layout, counts=counts, seed=19)


def test_forward_experts_with_unassigned_rows(mc):
    run_forward(mc, 400, 136, 264, "gelu", "kn", counts=[100, 0, 150], first=37, seed=23)
    run_forward(mc, 40, 136, 264, "gelu", "kn", counts=[10, 0, 15], first=3, seed=23)


def run_backward(mc, rows, K, N, act, layout, counts=None, first=0, dw="bf16", bias="bf16", extra=0, seed=0):
    E = len(counts) if counts is not None else 0
    lead = (E,) if E else ()
    X = draw((rows, K), 1.0, seed)
    W = draw(lead + ((K, N) if layout == "kn" else (N, K)), K ** -0.5, seed + 1)
    dY = draw((rows, N), 0.25, seed + 2)
    Z = draw((rows, N), 1.5, seed + 3) if act != "none" else None
    off = offsets_of(counts, first) if E else None
    bdt, wdt = (F32 if bias == "f32" else BF), (F32 if dw == "f32" else BF)
    dX = blank(rows, K, extra)
    dW = torch.full(W.shape, float("nan"), dtype=wdt, device=DEV)
    db = torch.full(lead + (N,), float("nan"), dtype=bdt, device=DEV)
    with mc.Linear(K, N, activation=act, experts=E, weight_layout=layout, bias_dtype=bdt, dw_dtype=wdt) as lin:
        ws = torch.full((max(lin.workspace_size(rows), 256),), 0xff, dtype=torch.uint8, device=DEV)   # NaNs
        args = (wide(dY, extra), wide(X, extra), W.to(DEV))
        kw = dict(Z=wide(Z, extra) if Z is not None else None, offsets=torch.from_numpy(off).to(DEV) if E else None,
                  workspace=ws)
        lin.backward(*args, dX=dX, dW=dW, dbias=db, **kw)
        assert lin.check() == 0
        # one at a time: the same bits
        dX2, dW2, db2 = blank(rows, K, 0), torch.empty_like(dW), torch.empty_like(db)
        lin.backward(*args, dX=dX2, **kw)
        lin.backward(*args, dW=dW2, **kw)
        lin.backward(*args, dbias=db2, **kw)
        assert lin.check() == 0
    (dx, sx), (dw_, sw), (db_, sb) = ref.linear_grad(f64(dY), f64(X), f64(W), f64(Z), act, layout, off)
    used = ~np.isnan(dx[:, 0])
    rnd = 2.0 ** -8 if act != "none" else 0.0          # dZ rounded for the products
    big = max((c for c in counts), default=0) if E else rows
    ut = torch.from_numpy(used)
    check_close(dX[ut], dx[used], (rnd + (N / 16 + 16) * 2.0 ** -22) * sx[used] + 2.0 ** -8 * np.abs(dx[used]), "dX")
    assert bool(torch.isnan(dX[~ut].float()).all())
    check_close(dW, dw_, (rnd + (big / 16 + 16) * 2.0 ** -22) * sw + (2.0 ** -8 if dw == "bf16" else 0) * np.abs(dw_), "dW")
    # at most `big` fp32 additions, and act' to 2^-18
    check_close(db, db_, (big * 2.0 ** -24 + 2.0 ** -18) * sb + 2.0 ** -18 * sb + (2.0 ** -8 if bias == "bf16" else 0) * np.abs(db_),
                "dbias")
    assert torch.equal(dX[ut], dX2[ut]) and torch.equal(dW, dW2) and torch.equal(db, db2)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("rows,K,N", [(1, 8, 8), (3, 264, 72), (50, 136, 520), (64, 128, 256), (129, 520, 264), (333, 1000, 200),
                                      (1000, 264, 1032)])
def test_backward_odd_sizes(mc, rows, K, N, layout):
    run_backward(mc, rows, K, N, "gelu", layout, seed=rows)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("dw,bias", [("f32", "f32"), ("bf16", "bf16")])
def test_backward_activations_and_types(mc, act, dw, bias):
    run_backward(mc, 210, 264, 328, act, "kn", dw=dw, bias=bias, extra=16, seed=29)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("layout,act", [("kn", "gelu"), ("nk", "none")])
def test_backward_experts(mc, counts, layout, act):
    run_backward(mc, max(sum(counts), 1), 264, 392, act, layout, counts=counts, seed=31)


def test_backward_experts_many_tiles(mc):
    """Many output tiles, with ragged tails in most experts."""
    counts = [100, 64, 0, 1, 200, 15, 129, 300]
    run_backward(mc, sum(counts), 2048, 2048, "silu", "kn", counts=counts, seed=37)
    run_backward(mc, 1000, 2048, 2048, "none", "nk", counts=counts, first=50, seed=38)


def test_poison_outside_a_group_stays_outside(mc):
    """NaN rows of one expert do not reach the others' outputs or gradients."""
    counts, K, N = [70, 50, 90], 136, 264
    off = offsets_of(counts)
    rows = sum(counts)
    X, W, dY = draw((rows, K), 1.0, 41), draw((3, K, N), K ** -0.5, 42), draw((rows, N), 1.0, 43)
    X[off[1]:off[2]] = float("nan")
    dY[off[1]:off[2]] = float("inf")
    with mc.Linear(K, N, experts=3) as lin:
        Y, dX, dW = blank(rows, N, 0), blank(rows, K, 0), torch.empty(3, K, N, dtype=BF, device=DEV)
        ws = torch.empty(max(lin.workspace_size(rows), 256), dtype=torch.uint8, device=DEV)
        o = torch.from_numpy(off).to(DEV)
        lin.forward(X.to(DEV), W.to(DEV), Y, offsets=o)
        lin.backward(dY.to(DEV), X.to(DEV), W.to(DEV), dX=dX, dW=dW, offsets=o, workspace=ws)
        assert lin.check() == 0
    for t in (Y, dX):
        good = torch.cat([t[:off[1]], t[off[2]:]])
        assert bool(torch.isfinite(good.float()).all())
    assert bool(torch.isfinite(dW[0].float()).all()) and bool(torch.isfinite(dW[2].float()).all())
    assert bool(torch.isnan(dW[1].float()).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_gradient_against_differences(mc, act):
    """<dW, U> and <dX, V> against central differences of the 64-bit loss sum(Y * G) along random directions."""
    rows, K, N = 96, 64, 72
    X, W, b, G = draw((rows, K), 1.0, 51), draw((K, N), K ** -0.5, 52), draw((N,), 0.5, 53), draw((rows, N), 1.0, 54)
    with mc.Linear(K, N, activation=act, bias_dtype=F32, dw_dtype=F32) as lin:
        Y, Z = blank(rows, N, 0), blank(rows, N, 0)
        dX, dW, db = blank(rows, K, 0), torch.empty(K, N, device=DEV), torch.empty(N, device=DEV)
        ws = torch.empty(lin.workspace_size(rows), dtype=torch.uint8, device=DEV)
        bd = b.float().to(DEV)
        lin.forward(X.to(DEV), W.to(DEV), Y, bias=bd, Z=Z)
        lin.backward(G.to(DEV), X.to(DEV), W.to(DEV), Z=Z, dX=dX, dW=dW, dbias=db, workspace=ws)
        assert lin.check() == 0
    x, w, bb, gg = f64(X), f64(W), f64(b), f64(G)

    def loss(x, w, bb):
        return float((ref.linear(x, w, bb, None, act, "kn", None)[0] * gg).sum())

    rng = np.random.default_rng(5)
    h = 1e-5
    # Z reaches the backward pass rounded to bf16 (2^-9 relative, slope of act' below 1.2 and |z| a few), dZ too:
    # each term of the inner product is off by 2^-7 of its size at most; relu's kink adds nothing at |z| > h.
    for got, arg, base in ((dX, 0, x), (dW, 1, w), (db, 2, bb)):
        U = rng.standard_normal(base.shape)
        args = [x, w, bb]
        up, dn = list(args), list(args)
        up[arg], dn[arg] = base + h * U, base - h * U
        num = (loss(*up) - loss(*dn)) / (2 * h)
        scale = np.abs(f64(got) * U).sum()
        assert abs(float((f64(got) * U).sum()) - num) <= 2.0 ** -6 * scale


def test_extreme_values_of_the_activations(mc):
    """An identity product carries the arguments: limits, infinities and NaN of act and act'."""
    vals = torch.tensor([0.0, -0.0, 1.0, -1.0, 8.0, -8.0, 30.0, -30.0, 1e4, -1e4, 3e38, -3e38, 1e-30, -1e-30, 0.5, float("nan")],
                        dtype=BF)
    n = 16
    X = torch.diag(torch.ones(n)).to(BF)
    for act in ("relu", "gelu", "silu"):
        with mc.Linear(n, n, activation=act) as lin:
            Y = blank(n, n, 0)
            lin.forward(X.to(DEV), torch.zeros(n, n, dtype=BF, device=DEV), Y, bias=vals.to(DEV))
            dW, db = torch.empty(n, n, dtype=BF, device=DEV), torch.empty(n, dtype=BF, device=DEV)
            ws = torch.empty(lin.workspace_size(n), dtype=torch.uint8, device=DEV)
            Zs = vals.to(DEV).expand(n, n).contiguous()
            one = torch.zeros(n, n, dtype=BF, device=DEV)
            one[0] = 1.0
            Zs[1:] = 0.0
            lin.backward(one, X.to(DEV), None, Z=Zs, dW=dW, dbias=db, workspace=ws)
            assert lin.check() == 0
        v = f64(vals)
        with np.errstate(over="ignore", invalid="ignore"):
            y, g = ref.act(act, v), ref.act_grad(act, np.clip(v, -1e6, 1e6))
        for j in range(n - 1):
            assert abs(f64(Y)[0, j] - y[j]) <= 2.0 ** -8 * abs(y[j]) + 1e-12, (act, v[j])
            assert abs(f64(db)[j] - g[j]) <= 2.0 ** -8 * abs(g[j]) + 2.0 ** -18, (act, v[j])
        assert np.isnan(f64(Y)[0, n - 1])
        if act != "relu":
            assert np.isnan(f64(db)[n - 1])


def test_repeated_runs_give_the_same_bits_on_two_streams(mc):
    """No atomics in the sums: two streams at once, each with its own buffers, repeat the first result."""
    rows, K, N = 300, 1032, 520
    X, W, dY, Z = (draw(s, 1.0, 60 + i).to(DEV) for i, s in enumerate([(rows, K), (K, N), (rows, N), (rows, N)]))
    with mc.Linear(K, N, activation="gelu") as lin:
        def call(stream):
            out = [blank(rows, N, 0), blank(rows, K, 0), torch.empty_like(W), torch.empty(N, dtype=BF, device=DEV)]
            ws = torch.empty(lin.workspace_size(rows), dtype=torch.uint8, device=DEV)
            lin.forward(X, W, out[0], stream=stream)
            lin.backward(dY, X, W, Z=Z, dX=out[1], dW=out[2], dbias=out[3], workspace=ws, stream=stream)
            return out, ws
        first, _ = call(None)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        keep = [call(streams[i % 2]) for i in range(6)]
        torch.cuda.synchronize()
        assert lin.check() == 0
        for out, _ in keep:
            assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_bad_offsets_are_clamped_and_reported(mc):
    rows, K, N = 100, 64, 64
    X, W = draw((rows, K), 1.0, 71).to(DEV), draw((2, K, N), 0.1, 72).to(DEV)
    Y = blank(rows, N, 0)
    with mc.Linear(K, N, experts=2) as lin:
        lin.forward(X, W, Y, offsets=torch.tensor([0, 120, 90], dtype=torch.int32, device=DEV))
        assert lin.check() == mc.ERR_INVALID_ARG
        lin.forward(X, W, Y, offsets=torch.tensor([0, 60, 100], dtype=torch.int32, device=DEV))
        assert lin.check() == 0
        assert bool(torch.isfinite(Y.float()).all())


def test_zero_rows(mc):
    K, N = 64, 72
    W = torch.ones(K, N, dtype=BF, device=DEV)
    e = lambda c: torch.empty(0, c, dtype=BF, device=DEV)
    dW, db = torch.ones_like(W), torch.ones(N, dtype=BF, device=DEV)
    with mc.Linear(K, N, activation="gelu") as lin:
        ws = torch.empty(max(lin.workspace_size(0), 256), dtype=torch.uint8, device=DEV)
        lin.forward(e(K), W, e(N))
        lin.backward(e(N), e(K), W, Z=e(N), dX=e(K), dW=dW, dbias=db, workspace=ws)
        assert lin.check() == 0
    assert not bool(dW.any()) and not bool(db.any())


def test_refusals_of_tensors(mc):
    K, N, rows = 64, 72, 10
    t = lambda *s, d=BF: torch.empty(*s, dtype=d, device=DEV)
    with mc.Linear(K, N, activation="gelu") as lin:
        X, W, Y = t(rows, K), t(K, N), t(rows, N)
        for bad in (dict(X=t(rows, K, d=F32)), dict(X=t(rows, K + 8)), dict(X=t(K, rows).t()), dict(W=t(N, K)), dict(Y=t(rows + 1, N)),
                    dict(Y=None)):
            a = dict(X=X, W=W, Y=Y)
            a.update(bad)
            with pytest.raises(ValueError):
                lin.forward(a["X"], a["W"], a["Y"])
        for kw in (dict(bias=t(N + 8)), dict(residual=t(rows, K)), dict(Z=t(rows, N, d=F32)), dict(offsets=t(2, d=torch.int32))):
            with pytest.raises(ValueError):
                lin.forward(X, W, Y, **kw)
        with pytest.raises(mc.MlpChainError):      # a row stride that is no multiple of 8
            lin.forward(t(rows, K + 4)[:, :K], W, Y)
        with pytest.raises(mc.MlpChainError):      # a base that is not 16-byte aligned
            lin.forward(t(rows, K + 8)[:, 4:4 + K], W, Y)
        with pytest.raises(ValueError):            # an activation's gradient needs Z
            lin.backward(Y, X, W, dX=X)
        with pytest.raises(mc.MlpChainError):      # ... and a workspace
            lin.backward(Y, X, W, Z=t(rows, N), dX=t(rows, K))
        with pytest.raises(ValueError):
            lin.backward(Y, X, W, Z=t(rows, N), dX=t(rows, K), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
        assert lin.check() == 0
    with mc.Linear(K, N, experts=4) as lin:
        with pytest.raises(ValueError):            # offsets are missing
            lin.forward(X, t(4, K, N), Y)
        with pytest.raises(ValueError):
            lin.forward(X, t(4, K, N), Y, offsets=t(4, d=torch.int32))


def test_pairs_with_an_odd_ring_keep_their_fills_apart(mc):
    """Products split over CTA pairs whose ring has an odd number of slots, many launches back to back: each has the first
    one's bits and none runs into a bounded wait."""
    found = 0
    for rows, K, N, E in ((384, 4096, 4096, 0), (380, 1544, 9224, 0), (430, 4104, 4096, 0), (200, 5896, 2056, 5), (700, 5896, 1032, 6),
                          (1000, 8200, 520, 7)):
        with mc.Linear(K, N, experts=E) as lin:
            p = lin.plan(rows)
            if p["cta_pair"] != 2 or p["pipe_stages"] % 2 == 0:
                continue
            found += p["k_split"] > 1
            X, W = draw((rows, K), 1.0, 80).to(DEV), draw(((E, K, N) if E else (K, N)), K ** -0.5, 81).to(DEV)
            off = torch.tensor([rows * i // E for i in range(E + 1)], dtype=torch.int32, device=DEV) if E else None
            first = blank(rows, N, 0)
            lin.forward(X, W, first, offsets=off)
            outs = [blank(rows, N, 0) for _ in range(4)]
            for i in range(60):
                lin.forward(X, W, outs[i % 4], offsets=off)
            assert lin.check() == 0, p
            assert all(torch.equal(first, o) for o in outs), p
            want = torch.cat([X[rows * i // E:rows * (i + 1) // E].float() @ W[i].float() for i in range(E)]) if E else X.float() @ W.float()
            assert float((first.float() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    assert found


WIDE = [(979, 2056, 5912, None), (394, 1544, 13208, None), (845, 1032, 9992, None), (1579, 2056, 2056, None), (301, 4104, 19000, None),
        (1800, 2056, 3448, [300, 0, 511, 513, 33, 443]), (2300, 1928, 3080, [1, 1200, 600, 499])]


def test_some_products_take_tiles_of_more_than_256_columns(mc):
    n = 0
    for rows, K, N, counts in WIDE:
        with mc.Linear(K, N, activation="gelu", experts=len(counts or ())) as lin:
            n += lin.plan(rows)["tile_cols"] > 256
    assert n >= 3


@pytest.mark.parametrize("rows,K,N,counts", WIDE)
def test_forward_tiles_of_more_than_256_columns(mc, rows, K, N, counts):
    run_forward(mc, rows, K, N, "gelu", "kn", counts=counts, extra=8 if rows % 2 else 0, seed=rows)


@pytest.mark.parametrize("rows,K,N,counts", [(979, 5912, 520, None), (1800, 3448, 264, [300, 0, 511, 513, 33, 443])])
def test_backward_tiles_of_more_than_256_columns(mc, rows, K, N, counts):
    run_backward(mc, rows, K, N, "gelu", "nk", counts=counts, seed=rows)

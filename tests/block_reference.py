"""64-bit definitions of the operators of an MLP block, on the CPU, for the tests (numpy only)."""
import numpy as np

C = np.sqrt(2.0 / np.pi)
A = 0.044715


def sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


def act(name, z):
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        return z * sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + np.tanh(C * (z + A * z ** 3)))
    return z


def act_grad(name, z):
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name == "silu":
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        t = np.tanh(C * (z + A * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C * (1.0 + 3.0 * A * z * z)
    return np.ones_like(z)


def groups(rows, offsets):
    if offsets is None:
        return [(None, 0, rows)]
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def linear(X, W, b, R, name, layout, offsets):
    """(Y, Z, S) with S = sum_k |x||w| + |b|, the scale of the accumulation error; rows of no group are NaN."""
    rows = X.shape[0]
    N = W.shape[-1] if layout == "kn" else W.shape[-2]
    Z, S = np.full((rows, N), np.nan), np.full((rows, N), np.nan)
    for e, lo, hi in groups(rows, offsets):
        w = W if e is None else W[e]
        w = w if layout == "kn" else w.T
        Z[lo:hi], S[lo:hi] = X[lo:hi] @ w, np.abs(X[lo:hi]) @ np.abs(w)
        if b is not None:
            bb = b if e is None else b[e]
            Z[lo:hi] += bb
            S[lo:hi] += np.abs(bb)
    Y = act(name, Z)
    return (Y if R is None else Y + R), Z, S


def linear_grad(dY, X, W, Z, name, layout, offsets):
    """dX, dW, db and the sums of absolute products behind each."""
    rows = X.shape[0]
    dZ = dY * (act_grad(name, Z) if Z is not None else 1.0)
    dX, sX = np.full(X.shape, np.nan), np.full(X.shape, np.nan)
    dW, sW = np.zeros(W.shape), np.zeros(W.shape)
    N = dY.shape[1]
    db, sb = np.zeros(W.shape[:-2] + (N,)), np.zeros(W.shape[:-2] + (N,))
    for e, lo, hi in groups(rows, offsets):
        w = W if e is None else W[e]
        wt = w.T if layout == "kn" else w
        dz, x = dZ[lo:hi], X[lo:hi]
        dX[lo:hi], sX[lo:hi] = dz @ wt, np.abs(dz) @ np.abs(wt)
        gw, gs = x.T @ dz, np.abs(x).T @ np.abs(dz)
        if layout == "nk":
            gw, gs = gw.T, gs.T
        if e is None:
            dW, sW, db, sb = gw, gs, dz.sum(0), np.abs(dz).sum(0)
        else:
            dW[e], sW[e], db[e], sb[e] = gw, gs, dz.sum(0), np.abs(dz).sum(0)
    return (dX, sX), (dW, sW), (db, sb)


def norm(x, gamma, beta, eps):
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (x - mean) * rstd
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean[:, 0], rstd[:, 0]


def norm_grad(dy, x, gamma, mean, rstd, add):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma if gamma is not None else dy
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return (dx if add is None else dx + add), (dy * xh).sum(0), dy.sum(0)

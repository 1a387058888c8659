"""CPU-only checks of the block operators' C ABI: exported symbols and bindings, struct layouts, refusals that are
decided before any CUDA call, and the 64-bit reference formulas against differences."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import block_reference as ref
import mlp_latency_gb300 as mc
from mlp_latency_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = 1, 2
INVALID, UNSUPPORTED = 1, 2
P = 1 << 20          # a plausible aligned address; nothing dereferences it


@pytest.fixture(scope="module")
def lib():
    mc.build()
    return mc.load()


def test_every_declared_symbol_has_an_export_and_a_binding(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mlp_block.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mlp_\w+)\s*\(", src)))
    assert len(names) == 10
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES, n


def test_struct_layouts_match_the_c_compiler(tmp_path):
    structs = {"mlp_linear_desc": _lib.LinearDesc, "mlp_linear_plan": _lib.LinearPlan}
    body = "".join(f'printf("{c} %zu\\n", sizeof({c}));' + "".join(
        f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in k._fields_) for c, k in structs.items())
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mlp_block.h"\nint main(void) {' + body + "return 0; }")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    sizes = dict(l.rsplit(" ", 1) for l in out.splitlines())
    for c, k in structs.items():
        assert int(sizes[c]) == ctypes.sizeof(k)
        for f, _ in k._fields_:
            assert int(sizes[f"{c}.{f}"]) == getattr(k, f).offset


def desc(**kw):
    d = dict(K=64, N=64, experts=0, weight_layout=0, activation=0, bias_dtype=BF, dw_dtype=BF, device=0, timeout_us=0)
    d.update(kw)
    return _lib.LinearDesc(*d.values())


@pytest.mark.parametrize("kw,want", [(dict(K=0), INVALID), (dict(K=60), INVALID), (dict(N=12), INVALID), (dict(N=-8), INVALID),
                                     (dict(K=1 << 31), INVALID), (dict(experts=-1), INVALID), (dict(experts=1025), INVALID),
                                     (dict(weight_layout=2), INVALID), (dict(device=-1), INVALID), (dict(activation=4), UNSUPPORTED),
                                     (dict(bias_dtype=0), UNSUPPORTED), (dict(dw_dtype=3), UNSUPPORTED)])
def test_linear_create_refuses(lib, kw, want):
    h = ctypes.c_void_p(5)
    assert lib.mlp_linear_create(ctypes.byref(desc(**kw)), ctypes.byref(h)) == want
    assert h.value is None


def test_linear_null_handles(lib):
    n = ctypes.c_size_t()
    assert lib.mlp_linear_create(None, None) == INVALID
    assert lib.mlp_linear_destroy(None) == INVALID
    assert lib.mlp_linear_workspace_size(None, 1, ctypes.byref(n)) == INVALID
    assert lib.mlp_linear_forward(None, 1, P, 64, P, None, None, 0, None, None, 0, P, 64, None) == INVALID
    assert lib.mlp_linear_backward(None, 1, P, 64, P, 64, P, None, 0, None, P, 64, None, None, None, None) == INVALID
    assert lib.mlp_linear_check(None, None) == INVALID
    assert lib.mlp_linear_get_plan(None, 1, 0, None) == INVALID


def fwd(lib, rows=4, cols=64, x=P, ldx=64, dt=BF, gamma=P, beta=P, wdt=BF, eps=1e-5, y=P, ldy=64, mean=None, rstd=None):
    return lib.mlp_layernorm_forward(rows, cols, x, ldx, dt, gamma, beta, wdt, eps, y, ldy, mean, rstd, None)


@pytest.mark.parametrize("kw,want", [(dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(rows=1 << 31), INVALID),
                                     (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=P + 1), INVALID),
                                     (dict(ldx=63), INVALID), (dict(ldy=63), INVALID), (dict(eps=-1.0), INVALID),
                                     (dict(eps=float("nan")), INVALID), (dict(gamma=P + 1), INVALID), (dict(mean=P + 2), INVALID),
                                     (dict(dt=0), UNSUPPORTED), (dict(wdt=7), UNSUPPORTED), (dict(rows=0), 0)])
def test_layer_norm_forward_refuses(lib, kw, want):
    assert fwd(lib, **kw) == want


def bwd(lib, rows=4, cols=64, dy=P, lddy=64, x=P, ldx=64, dt=BF, gamma=P, wdt=BF, mean=P, rstd=P, add=None, ldadd=0, dx=P, lddx=64,
        dgamma=None, dbeta=None, ws=None):
    return lib.mlp_layernorm_backward(rows, cols, dy, lddy, x, ldx, dt, gamma, wdt, mean, rstd, add, ldadd, dx, lddx, dgamma, dbeta,
                                      ws, None)


@pytest.mark.parametrize("kw,want", [(dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dy=None), INVALID), (dict(x=None), INVALID),
                                     (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(lddy=60), INVALID),
                                     (dict(lddx=60), INVALID), (dict(add=P, ldadd=8), INVALID), (dict(dgamma=P), INVALID),
                                     (dict(dbeta=P, ws=P + 16), INVALID), (dict(dgamma=P + 1, ws=P), INVALID),
                                     (dict(dx=P + 1), INVALID), (dict(dt=5), UNSUPPORTED), (dict(wdt=0), UNSUPPORTED)])
def test_layer_norm_backward_refuses(lib, kw, want):
    assert bwd(lib, **kw) == want


def test_layer_norm_workspace(lib):
    assert mc.layer_norm_workspace_size(100, 64) >= 2 * 64 * 4
    n = ctypes.c_size_t()
    assert lib.mlp_layernorm_workspace_size(-1, 64, ctypes.byref(n)) == INVALID
    assert lib.mlp_layernorm_workspace_size(1, 0, ctypes.byref(n)) == INVALID
    assert lib.mlp_layernorm_workspace_size(1, 1, None) == INVALID


def test_python_refuses_unknown_options():
    for kw in (dict(activation="tanh"), dict(weight_layout="nn"), dict(bias_dtype=None), dict(dw_dtype=int)):
        with pytest.raises(ValueError):
            mc.Linear(64, 64, **kw)


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
def test_reference_activation_gradients_against_differences(name):
    z = np.linspace(-6, 6, 241) + 0.0123
    h = 1e-6
    num = (ref.act(name, z + h) - ref.act(name, z - h)) / (2 * h)
    assert np.abs(num - ref.act_grad(name, z)).max() < 1e-8


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_reference_linear_gradients_against_differences(layout):
    rng = np.random.default_rng(1)
    off = [0, 3, 3, 7]
    X, W, b = rng.standard_normal((7, 5)), rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 4))
    if layout == "nk":
        W = np.ascontiguousarray(W.transpose(0, 2, 1))
    G = rng.standard_normal((7, 4))
    Z = ref.linear(X, W, b, None, "gelu", layout, off)[1]
    (dX, _), (dW, _), (db, _) = ref.linear_grad(G, X, W, Z, "gelu", layout, off)
    assert not dW[1].any() and not db[1].any()
    h = 1e-6
    for got, i in ((dX, 0), (dW, 1), (db, 2)):
        a = [X, W, b]
        U = rng.standard_normal(a[i].shape)
        up, dn = list(a), list(a)
        up[i], dn[i] = a[i] + h * U, a[i] - h * U
        num = ((ref.linear(*up, None, "gelu", layout, off)[0] - ref.linear(*dn, None, "gelu", layout, off)[0]) * G).sum() / (2 * h)
        assert abs(num - (got * U).sum()) < 1e-6 * (1 + abs(num))


def test_reference_norm_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, g, b, G = rng.standard_normal((4, 9)) * 2, rng.standard_normal(9), rng.standard_normal(9), rng.standard_normal((4, 9))
    _, m, r = ref.norm(x, g, b, 1e-5)
    grads = ref.norm_grad(G, x, g, m, r, None)
    h = 1e-6
    for i, got in enumerate(grads):
        a = [x, g, b]
        U = rng.standard_normal(a[i].shape)
        up, dn = list(a), list(a)
        up[i], dn[i] = a[i] + h * U, a[i] - h * U
        num = ((ref.norm(*up, 1e-5)[0] - ref.norm(*dn, 1e-5)[0]) * G).sum() / (2 * h)
        assert abs(num - (got * U).sum()) < 1e-6 * (1 + abs(num))


def test_layer_norm_refuses_tensors_before_any_launch(lib):
    x, w = torch.zeros(2, 8), torch.zeros(8)
    v = torch.zeros(2)
    for call, what in ((lambda: mc.layer_norm_forward(x, w, w, x), "x: expected a CUDA tensor"),
                       (lambda: mc.layer_norm_forward(None, w, w, x), "x is missing"),
                       (lambda: mc.layer_norm_forward([1.0], w, w, x), "x: expected a tensor"),
                       (lambda: mc.layer_norm_forward(w, w, w, x), "layer norm takes matrices"),
                       (lambda: mc.layer_norm_forward(x.int(), w, w, x), "layer norm takes matrices"),
                       (lambda: mc.layer_norm_forward(x, w.half(), None, x), "layer norm weights are"),
                       (lambda: mc.layer_norm_backward(None, x, w, v, v, x), "dy is missing")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        mc.layer_norm_forward(x, w, w)

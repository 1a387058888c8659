"""CPU-only checks of routing, of the exchange of rows and of clipping: exported symbols and bindings, struct layout,
refusals that are decided before any CUDA call, and the 64-bit reference formulas against differences."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import experts_reference as ref
import mlp_latency_gb300 as mc
from mlp_latency_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 1 << 20          # a plausible aligned address; nothing dereferences it
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    mc.build()
    return mc.load()


@pytest.mark.parametrize("header,count", [("mlp_experts.h", 7), ("mlp_clip.h", 3)])
def test_every_declared_symbol_has_an_export_and_a_binding(lib, header, count):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mlp_\w+)\s*\(", src)))
    assert len(names) == count
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES, n


def test_the_headers_compile_as_c_and_the_struct_layout_matches(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mlp_experts.h"\n#include "mlp_clip.h"\nint main(void) {'
                   'printf("%zu %zu %zu %zu %zu", sizeof(mlp_tensor), offsetof(mlp_tensor, data), offsetof(mlp_tensor, out),'
                   'offsetof(mlp_tensor, count), offsetof(mlp_tensor, dtype)); return 0; }')
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    k = _lib.Tensor
    assert out.split() == [str(v) for v in (ctypes.sizeof(k), k.data.offset, k.out.offset, k.count.offset, k.dtype.offset)]


# ------------------------------------------------------------------------------------ refusals --
def route(lib, tokens=4, experts=8, top=2, logits=P, ldl=8, dt=F32, mask=None, gates=P, chosen=P, slots=P, offsets=P, counts=None, loss=None,
          ws=P):
    return lib.mlp_route_forward(tokens, experts, top, logits, ldl, dt, mask, 0, gates, chosen, slots, offsets, counts, loss, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(experts=0), INVALID), (dict(experts=1025, ldl=1025), INVALID), (dict(top=0), INVALID),
    (dict(top=9), INVALID), (dict(experts=64, ldl=64, top=33), INVALID), (dict(tokens=1 << 30), INVALID), (dict(logits=None), INVALID),
    (dict(logits=P + 2), INVALID), (dict(ldl=7), INVALID), (dict(gates=None), INVALID), (dict(gates=P + 2), INVALID),
    (dict(chosen=None), INVALID), (dict(slots=None), INVALID), (dict(slots=P + 1), INVALID), (dict(offsets=None), INVALID),
    (dict(offsets=P + 2), INVALID), (dict(counts=P + 2), INVALID), (dict(loss=P + 1), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 128), INVALID), (dict(dt=0), UNSUPPORTED), (dict(dt=3), UNSUPPORTED)])
def test_route_forward_refuses(lib, kw, want):
    assert route(lib, **kw) == want


def route_back(lib, tokens=4, experts=8, top=2, logits=P, ldl=8, dt=F32, chosen=P, offsets=P, dgates=P, dloss=P, dlogits=P, ldd=8):
    return lib.mlp_route_backward(tokens, experts, top, logits, ldl, dt, 0, chosen, offsets, dgates, dloss, dlogits, ldd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(experts=2000), INVALID), (dict(top=9), INVALID), (dict(logits=None), INVALID),
    (dict(dlogits=None), INVALID), (dict(dlogits=P + 1), INVALID), (dict(ldd=7), INVALID), (dict(chosen=None), INVALID),
    (dict(offsets=None), INVALID), (dict(dgates=P + 1), INVALID), (dict(dloss=P + 2), INVALID), (dict(dt=7), UNSUPPORTED),
    (dict(tokens=0), OK)])
def test_route_backward_refuses(lib, kw, want):
    assert route_back(lib, **kw) == want


def test_workspaces(lib):
    n = ctypes.c_size_t()
    for bad in ((-1, 8), (8, 0), (8, 1025)):
        assert lib.mlp_route_workspace_size(*bad, ctypes.byref(n)) == INVALID
    assert lib.mlp_route_workspace_size(1, 8, None) == INVALID
    assert lib.mlp_clip_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert lib.mlp_clip_workspace_size(1, None) == INVALID
    assert mc.clip_workspace_size(5000) > mc.clip_workspace_size(1) > 0
    with pytest.raises(mc.MlpChainError):
        mc.route_workspace_size(4, 0)


def call(lib, what, tokens=4, cols=64, top=2, a=P, lda=64, dt=BF, slots=P, rows=8, b=P, ldb=64, add=None, ldadd=64, gates=P, dgates=P):
    if what == "dispatch_forward":
        return lib.mlp_dispatch_forward(tokens, cols, top, a, lda, dt, slots, rows, b, ldb, None)
    if what == "dispatch_backward":
        return lib.mlp_dispatch_backward(tokens, cols, top, a, lda, dt, slots, rows, add, ldadd, b, ldb, None)
    if what == "combine_forward":
        return lib.mlp_combine_forward(tokens, cols, top, a, lda, dt, gates, slots, rows, add, ldadd, b, ldb, None)
    return lib.mlp_combine_backward(tokens, cols, top, a, lda, P, 64, dt, gates, slots, rows, b, ldb, dgates, None)


EXCHANGES = ("dispatch_forward", "dispatch_backward", "combine_forward", "combine_backward")


@pytest.mark.parametrize("what", EXCHANGES)
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=1 << 31), INVALID), (dict(top=0), INVALID), (dict(top=33), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(tokens=1 << 30), INVALID), (dict(a=None), INVALID), (dict(a=P + 1), INVALID),
    (dict(lda=63), INVALID), (dict(b=P + 1), INVALID), (dict(ldb=63), INVALID), (dict(slots=None), INVALID), (dict(slots=P + 2), INVALID),
    (dict(dt=0), UNSUPPORTED), (dict(dt=3), UNSUPPORTED), (dict(tokens=0), OK)])
def test_exchange_refuses(lib, what, kw, want):
    assert call(lib, what, **kw) == want


@pytest.mark.parametrize("what,kw,want", [
    ("dispatch_forward", dict(b=None), INVALID), ("dispatch_forward", dict(rows=0, b=None), OK), ("dispatch_backward", dict(b=None), INVALID),
    ("dispatch_backward", dict(add=P, ldadd=8), INVALID), ("dispatch_backward", dict(add=P + 1), INVALID),
    ("combine_forward", dict(gates=None), INVALID), ("combine_forward", dict(gates=P + 2), INVALID), ("combine_forward", dict(b=None), INVALID),
    ("combine_forward", dict(add=P, ldadd=63), INVALID), ("combine_backward", dict(gates=None), INVALID),
    ("combine_backward", dict(dgates=P + 2), INVALID), ("combine_backward", dict(b=None, dgates=None), OK)])
def test_an_exchange_refuses(lib, what, kw, want):
    assert call(lib, what, **kw) == want


def test_the_most_choices(lib):
    """tokens * top up to 2^31 - 1, whether top divides it or not.  (Sizes are looked at before the type, and that before anything else.)"""
    for top in (1, 2, 3, 5, 7, 31, 32):
        most = ((1 << 31) - 1) // top
        for tokens, want in ((most, UNSUPPORTED), (most + 1, INVALID)):
            assert route(lib, tokens=tokens, top=top, experts=64, ldl=64, dt=0) == want
            assert route_back(lib, tokens=tokens, top=top, experts=64, ldl=64, ldd=64, dt=0) == want
            for what in EXCHANGES:
                assert call(lib, what, tokens=tokens, top=top, dt=0) == want


@pytest.mark.parametrize("what", EXCHANGES)
def test_the_largest_exchanges_are_refused(lib, what):
    """Tokens times a row's pieces of 128 bytes from 2^31 on."""
    assert call(lib, what, tokens=1 << 26, cols=64 * 32, lda=64 * 32, ldb=64 * 32) == INVALID
    assert call(lib, what, tokens=1 << 26, cols=32 * 31 + 1, lda=64 * 32, ldb=64 * 32, dt=F32) == INVALID


def clip(lib, spans, max_norm=1.0, eps=1e-6, norm=P, ws=P, clipped=True, count=None):
    """spans: (data, out, elements, dtype)"""
    a = (_lib.Tensor * max(len(spans), 1))(*(_lib.Tensor(*s) for s in spans))
    n = len(spans) if count is None else count
    return lib.mlp_clip_gradients(n, a, max_norm, eps, norm, ws, None) if clipped else lib.mlp_gradient_norm(n, a, norm, ws, None)


ONE = (P, P, 100, BF)


@pytest.mark.parametrize("kw,want", [
    (dict(count=-1), INVALID), (dict(count=1 << 21), INVALID), (dict(norm=None), INVALID), (dict(norm=P + 2), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 64), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=NAN), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(spans=[(None, P, 4, BF)]), INVALID), (dict(spans=[(P + 1, P + 1, 4, BF)]), INVALID),
    (dict(spans=[(P + 2, P + 2, 4, F32)]), INVALID), (dict(spans=[(P, None, 4, BF)]), INVALID), (dict(spans=[(P, P + 1, 4, BF)]), INVALID),
    (dict(spans=[(P, P, -1, BF)]), INVALID), (dict(spans=[(P, P, 1 << 40, BF)]), INVALID), (dict(spans=[(P, P, 4, 0)]), UNSUPPORTED),
    (dict(spans=[ONE, ONE]), INVALID),                                              # the same tensor twice
    (dict(spans=[ONE, (P + 198, P + 198, 4, BF)]), INVALID),                        # its last element again
    (dict(spans=[(P, P + 2, 100, BF)]), INVALID),                                   # over its own data, shifted
    (dict(spans=[(P, P + 4096, 100, BF), (P + 4096, P + 8192, 100, BF)]), INVALID),  # over another's data
    (dict(spans=[(P, P + 4096, 100, BF), (P + 512, P + 4098, 100, BF)]), INVALID),  # two outs
    (dict(spans=[(P + 8192, P + 8192, 9, F32), (P, P, 5000, BF)]), INVALID)])       # out of order
def test_clip_refuses(lib, kw, want):
    kw = {"spans": [ONE], **kw}
    assert clip(lib, **kw) == want


def test_norm_refuses(lib):
    assert clip(lib, [(P + 1, None, 4, BF)], clipped=False) == INVALID
    assert clip(lib, [(P, None, 4, 9)], clipped=False) == UNSUPPORTED
    assert clip(lib, [ONE], norm=None, clipped=False) == INVALID


def test_python_refuses_before_any_launch(lib):
    x, i = torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)
    g, o, n = torch.zeros(2, 2), torch.zeros(9, dtype=torch.int32), torch.zeros(1)
    for call_, what in (
            (lambda: mc.route_forward(x, g, i, o, slots=i), "logits: expected a CUDA tensor"),
            (lambda: mc.route_forward(None, g, i, o, slots=i), "logits is missing"),
            (lambda: mc.route_forward(x.half(), g, i, o, slots=i), "route: logits is a matrix of"),
            (lambda: mc.route_forward(x, g, i[0], o, slots=i), "experts: expected int32"),
            (lambda: mc.route_forward(x, g, torch.zeros(2, 33, dtype=torch.int32), o, slots=i), "top 1 to 32"),
            (lambda: mc.route_backward(x, i, o, x), "logits: expected a CUDA tensor"),
            (lambda: mc.dispatch_forward(x, i, x), "x: expected a CUDA tensor"),
            (lambda: mc.dispatch_forward(x, i, n), "y: expected a matrix"),
            (lambda: mc.dispatch_backward(x, i, n), "dispatch: dx is a matrix"),
            (lambda: mc.combine_forward(x, g, i, x), "y: expected a CUDA tensor"),
            (lambda: mc.combine_backward(x, x, g, i, dz=x), "dy: expected a CUDA tensor"),
            (lambda: mc.gradient_norm([x], n), "norm: expected a contiguous CUDA tensor"),
            (lambda: mc.gradient_norm(x, n), "grads: expected a list or tuple"),
            (lambda: mc.clip_gradients(iter([x]), 1.0, n), "grads: expected a list or tuple")):
        with pytest.raises(ValueError, match=what):
            call_()


# ----------------------------------------------------------------------- the reference itself --
@pytest.mark.parametrize("normalize", [False, True])
def test_reference_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(3)
    l, mask = rng.standard_normal((7, 6)) * 1.5, np.array([1, 1, 0, 1, 1, 1, 1], bool)
    l[1, 2:] = -np.inf      # one with fewer experts than choices
    l[4] = -np.inf
    chosen = ref.choose(l, 3, mask)
    _, counts, _ = ref.rows_of(chosen, 6)
    assert list(chosen[2]) == [-1] * 3 and list(chosen[4]) == [-1] * 3 and chosen[1, 2] == -1
    G, c = rng.standard_normal((7, 3)), 0.7
    got = ref.route_grad(l, chosen, counts, G, c, normalize)[0]
    f = lambda a: (np.where(chosen >= 0, ref.gates_of(a, chosen, normalize), 0.0) * G).sum() + c * ref.loss_of(a, chosen, counts)[0]
    U, h = rng.standard_normal(l.shape), 1e-6
    num = (f(l + h * U) - f(l - h * U)) / (2 * h)
    assert abs(num - (got * U).sum()) < 1e-7 * (1 + abs(num))


def test_reference_loss_is_one_in_balance():
    l = np.zeros((8, 4))
    chosen = np.stack([np.arange(8) % 4, (np.arange(8) + 1) % 4], axis=1)
    _, counts, offsets = ref.rows_of(chosen, 4)
    assert list(counts) == [4] * 4 and offsets[-1] == 16
    assert abs(ref.loss_of(l, chosen, counts)[0] - 1.0) < 1e-15


def test_reference_exchange_is_its_own_transpose():
    rng = np.random.default_rng(5)
    chosen = ref.choose(rng.standard_normal((9, 4)), 2, np.arange(9) < 7)
    slots, _, offsets = ref.rows_of(chosen, 4)
    z, dy, gates = rng.standard_normal((18, 3)), rng.standard_normal((9, 3)), rng.random((9, 2))
    y = ref.gather(z, slots, gates, None)[0]
    dz = ref.scatter(np.zeros_like(z), dy, slots, gates)
    assert abs((y * dy).sum() - (z * dz).sum()) < 1e-12
    dg = ref.gate_grad(dy, z, slots)[0]
    U, h = rng.standard_normal(gates.shape), 1e-6
    num = ((ref.gather(z, slots, gates + h * U, None)[0] - ref.gather(z, slots, gates - h * U, None)[0]) * dy).sum() / (2 * h)
    assert abs(num - (dg * U).sum()) < 1e-7
    assert not dz[offsets[-1]:].any()

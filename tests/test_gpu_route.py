"""GPU tests of routing and its gradient against the 64-bit definitions.

Choices, rows, counts and offsets are whole numbers and equal.  Units are 2^-24, relative.  A p: expf is off by 2 of them
(1 ulp), the difference before it by |l - max| units of the result, the sum by an addition a lane's value and 5 shuffles
(and the terms' own errors, weighted by their p), the quotient by 1.  A loss sums p over tokens: a warp's in order, then
the warps' of a block, then the blocks'."""
import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
DEV, BF, F32, I32 = "cuda", torch.bfloat16, torch.float32, torch.int32
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
LOWEST = torch.finfo(F32).min


@pytest.fixture(scope="module")
def mc():
    import mlp_latency_gb300
    mlp_latency_gb300.build()
    return mlp_latency_gb300


def cdiv(a, b):
    return -(-a // b)


def logits_for(T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g)).to(dtype)


def forward(mc, logits, k, mask=None, normalize=False, extras=True, spoil=None):
    """Outputs with guards around them: a word before and after each, which must stay."""
    T, E = logits.shape
    guards = []

    def guarded(n, dtype):
        t = torch.full((n + 8,), 77, dtype=dtype, device=DEV)
        guards.append(t)
        return t[4:4 + n]

    out = {"gates": guarded(T * k, F32).view(T, k), "experts": guarded(T * k, I32).view(T, k), "slots": guarded(T * k, I32).view(T, k),
           "offsets": guarded(E + 1, I32)}
    if extras:
        out["counts"], out["loss"] = guarded(E, I32), guarded(1, F32)
    ws = torch.full((max(mc.route_workspace_size(T, E), 1),), 255, dtype=torch.uint8, device=DEV)
    mc.route_forward(logits, out["gates"], out["experts"], out["offsets"], slots=out["slots"], counts=out.get("counts"),
                     loss=out.get("loss"), mask=mask, normalize=normalize, workspace=ws)
    torch.cuda.synchronize()
    for g in guards:
        assert (g[:4] == 77).all() and (g[-4:] == 77).all()
    return {n: t.clone() for n, t in out.items()}


def p_units(l, chosen, normalize):
    """Error of a gate and of a p, in units, per choice and per token: what is given above."""
    E, k = l.shape[1], chosen.shape[1]
    with np.errstate(all="ignore"):
        d = np.where(l == -np.inf, 0.0, l.max(1, keepdims=True) - l)
    p = ref.softmax(l)
    spread = (p * d).sum(1)
    own = np.take_along_axis(d, np.maximum(chosen, 0), 1)
    return own + spread[:, None] + 4 + (k if normalize else cdiv(E, 32)) + 5 + 2, spread + np.where(p > 0, p * d, 0).max(1) + 4 + cdiv(E, 32) + 7


def check(mc, l, k, mask=None, normalize=False, extras=True):
    got = forward(mc, l.to(DEV) if not l.is_cuda else l, k, mask.to(DEV) if mask is not None else None, normalize, extras)
    T, E = l.shape
    l64 = l.cpu().double().numpy()
    chosen = ref.choose(l64, k, None if mask is None else mask.numpy())
    slots, counts, offsets = ref.rows_of(chosen, E)
    assert np.array_equal(got["experts"].cpu().numpy(), chosen)
    assert np.array_equal(got["slots"].cpu().numpy(), slots)
    assert np.array_equal(got["offsets"].cpu().numpy(), offsets)
    routed = np.where((chosen >= 0).any(1, keepdims=True), l64, -np.inf)
    want, (units, p_unit) = ref.gates_of(routed, chosen, normalize), p_units(routed, chosen, normalize)
    err = np.abs(got["gates"].cpu().double().numpy() - want)
    assert (err <= units * U * want + 2.0 ** -126).all(), float((err / np.maximum(want, 1e-300)).max() / U)
    if extras:
        assert np.array_equal(got["counts"].cpu().numpy(), counts)
        loss, _ = ref.loss_of(routed, chosen, counts)
        adds = cdiv(T, 8 * 304) + 32 + cdiv(304, 32) + 5 + cdiv(E, 32) + 5 + 8
        assert abs(float(got["loss"]) - loss) <= (float(p_unit.max(initial=0)) + adds) * U * loss
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (2, 7, 7), (3, 1024, 32), (17, 33, 5), (31, 64, 32), (32, 8, 2), (33, 8, 2), (257, 100, 6),
                                   (300, 256, 8), (1001, 16, 4), (2048, 8, 2), (2433, 5, 3), (2600, 300, 3), (5000, 40, 1), (700, 1000, 9)])
def test_forward(mc, T, E, k, dtype):
    for normalize in (False, True):
        check(mc, logits_for(T, E, dtype, T + E), k, normalize=normalize)


@pytest.mark.parametrize("T", [1, 9, 40, 2500])
def test_no_extras_and_padding(mc, T):
    g = torch.Generator().manual_seed(T)
    mask = torch.rand(T, generator=g) < 0.6
    check(mc, logits_for(T, 20, F32, T), 3, mask, extras=False)
    check(mc, logits_for(T, 20, BF, T), 3, mask, normalize=True)
    check(mc, logits_for(T, 20, F32, T), 3, torch.zeros(T, dtype=torch.bool))
    check(mc, logits_for(T, 20, F32, T), 3, torch.arange(T) < T - T // 3)


@pytest.mark.parametrize("T", [30, 600])
@pytest.mark.parametrize("normalize", [False, True])
def test_logits_without_a_value(mc, T, normalize):
    """-inf is never chosen; rows of nothing else choose nothing; the lowest finite value is a value."""
    l = logits_for(T, 37, F32, 5)
    l[torch.rand(l.shape, generator=torch.Generator().manual_seed(1)) < 0.5] = -INF
    l[3] = -INF
    l[T // 2, 1:] = -INF
    l[5], l[6, :] = LOWEST, LOWEST
    l[6, 11] = 0.0
    l[7] = 0.0
    got = check(mc, l, 6, normalize=normalize)
    assert got["experts"][5].tolist() == list(range(6)) and got["experts"][6].tolist() == [11, 0, 1, 2, 3, 4]
    check(mc, torch.full((T, 9), -INF), 4, normalize=normalize)


def test_ties_go_to_the_first(mc):
    l = torch.randint(-2, 3, (900, 70), generator=torch.Generator().manual_seed(2)).float()
    l[l == 0] = torch.where(torch.rand(int((l == 0).sum()), generator=torch.Generator().manual_seed(3)) < 0.5, 0.0, -0.0)
    check(mc, l, 9)
    check(mc, l.to(BF), 9, normalize=True)
    check(mc, torch.zeros(50, 200), 32)


def test_nan_and_infinity_come_first_and_show(mc):
    l = logits_for(40, 12, F32, 9)
    l[4, 7] = NAN
    l[4, 3] = INF
    l[9, 5] = INF
    l[9, 2] = INF
    got = forward(mc, l.to(DEV), 3)
    want = ref.choose(l.double().numpy(), 3, None)
    assert np.array_equal(got["experts"].cpu().numpy(), want) and want[4, 0] == 7 and want[4, 1] == 3 and list(want[9, :2]) == [2, 5]
    assert np.array_equal(got["slots"].cpu().numpy(), ref.rows_of(want, 12)[0])
    bad = torch.isnan(got["gates"]).any(1).cpu()
    assert bad.nonzero()[:, 0].tolist() == [4, 9] and torch.isnan(got["loss"]).all()


def test_rows_of_a_wider_matrix_and_odd_places(mc):
    for dtype in (F32, BF):
        wide = logits_for(333, 61, dtype, 1).to(DEV)
        l = wide[:, 3:44]
        got, want = forward(mc, l, 5), forward(mc, l.contiguous(), 5)
        assert all(torch.equal(got[n], want[n]) for n in got)
        check(mc, l, 5)


def test_no_tokens(mc):
    got = forward(mc, torch.empty(0, 6, device=DEV), 2)
    assert not got["offsets"].any() and not got["counts"].any() and float(got["loss"]) == 0.0


def test_more_than_there_is_is_refused(mc):
    e = lambda *s, d=F32: torch.empty(*s, dtype=d, device=DEV)
    for T, E, k in ((4, 2, 3), (4, 1025, 2)):
        with pytest.raises(mc.MlpChainError):
            mc.route_forward(e(T, E), e(T, k), e(T, k, d=I32), e(E + 1, d=I32), slots=e(T, k, d=I32), workspace=e(1 << 20, d=torch.uint8))
        with pytest.raises(mc.MlpChainError):
            mc.route_backward(e(T, E), e(T, k, d=I32), e(E + 1, d=I32), e(T, E))
    with pytest.raises(ValueError):
        mc.route_forward(e(4, 8), e(4, 2), e(4, 2, d=I32), e(9, d=I32), slots=e(4, 2, d=I32), workspace=e(16, d=torch.uint8))
    with pytest.raises(mc.MlpChainError):
        mc.route_forward(e(4, 8), e(4, 2), e(4, 2, d=I32), e(9, d=I32), slots=e(4, 2, d=I32))


def test_results_repeat(mc):
    l = logits_for(4000, 130, F32, 4).to(DEV)
    first = forward(mc, l, 4)
    for _ in range(5):
        again = forward(mc, l, 4)
        assert all(torch.equal(first[n], again[n]) for n in first)


# ------------------------------------------------------------------------------------ gradient --
def gradient(mc, l, k, normalize, mask=None, dgates=True, dloss=0.3, in_place=False):
    T, E = l.shape
    fw = forward(mc, l.to(DEV), k, mask.to(DEV) if mask is not None else None, normalize)
    G = torch.randn(T, k, generator=torch.Generator().manual_seed(T + k)) if dgates else None
    src = l.to(DEV).clone()
    out = src if in_place else torch.full_like(src, NAN)
    mc.route_backward(src, fw["experts"], fw["offsets"], out, dgates=G.to(DEV) if dgates else None,
                      dloss=torch.full((1,), dloss, device=DEV) if dloss is not None else None, normalize=normalize)
    chosen, counts = fw["experts"].cpu().long().numpy(), fw["counts"].cpu().double().numpy()
    l64 = np.where((chosen >= 0).any(1, keepdims=True), l.double().numpy(), -np.inf)
    c = float(torch.tensor(dloss if dloss is not None else 0.0, dtype=F32))
    want, size = ref.route_grad(l64, chosen, counts, G.double().numpy() if dgates else np.zeros((T, k)), c, normalize)
    units = sum(u.max(initial=0) for u in p_units(l64, chosen, normalize)) + 2 * (cdiv(E, 32) + 5) + k + 16
    got = out.cpu().double().numpy()
    err = np.abs(got - want)
    half = U if l.dtype == F32 else 2.0 ** -8
    tol = units * U * size + half * (np.abs(want) + units * U * size) + 2.0 ** -126
    assert (err <= tol).all(), float((err / tol).max())
    return out


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 1024, 32), (17, 33, 5), (300, 256, 8), (1001, 16, 4), (2048, 8, 2), (77, 500, 3)])
def test_gradient(mc, T, E, k, dtype, normalize):
    gradient(mc, logits_for(T, E, dtype, T + E), k, normalize)


@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_parts_padding_and_places(mc, normalize):
    l = logits_for(500, 24, F32, 7)
    l[torch.rand(l.shape, generator=torch.Generator().manual_seed(1)) < 0.4] = -INF
    l[3] = -INF
    l[9, 1:] = -INF
    mask = torch.arange(500) < 450
    for kw in (dict(dgates=False), dict(dloss=None), dict(dgates=False, dloss=None), dict(mask=mask), dict(in_place=True)):
        out = gradient(mc, l, 4, normalize, **kw)
        assert not out[3].any()
        if "mask" in kw:
            assert not out[450:].any()


def test_gradient_in_a_wider_matrix(mc):
    l = logits_for(100, 24, BF, 3).to(DEV)
    fw = forward(mc, l, 3)
    want, wide = torch.empty_like(l), torch.full((100, 31), 7.0, dtype=BF, device=DEV)
    G = torch.randn(100, 3, device=DEV)
    mc.route_backward(l, fw["experts"], fw["offsets"], want, dgates=G)
    mc.route_backward(l, fw["experts"], fw["offsets"], wide[:, 5:29], dgates=G)
    assert torch.equal(wide[:, 5:29], want) and (wide[:, :5] == 7).all() and (wide[:, 29:] == 7).all()


def test_choices_outside_the_experts_are_none(mc):
    l = logits_for(20, 8, F32, 3).to(DEV)
    fw = forward(mc, l, 3)
    chosen = fw["experts"].clone()
    chosen[4, 1], chosen[5, 2], none = 8, 1 << 30, chosen.clone()
    none[4, 1], none[5, 2] = -1, -1
    G, a, b = torch.randn(20, 3, device=DEV), torch.empty_like(l), torch.empty_like(l)
    mc.route_backward(l, chosen, fw["offsets"], a, dgates=G)
    mc.route_backward(l, none, fw["offsets"], b, dgates=G)
    assert torch.equal(a, b)


# ------------------------------------------------------------------------------ far and long calls --
def by_sorting(l, k, mask=None):
    """choices, slots and offsets of many tokens, by stable sorts on the CPU."""
    v, e = torch.sort(l.double(), dim=1, descending=True, stable=True)
    chosen = torch.where(v[:, :k] == -INF, -1, e[:, :k])
    if mask is not None:
        chosen[~mask] = -1
    flat, E = chosen.reshape(-1), l.shape[1]
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel())
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    return chosen, torch.where(flat < 0, -1, slots).view(chosen.shape), torch.cat([counts.new_zeros(1), counts.cumsum(0)])


@pytest.mark.parametrize("T,E,k,dtype", [(200001, 8, 8, F32), (123000, 8, 8, BF), (300000, 5, 2, F32), (17000, 1024, 32, BF), (60000, 33, 20, F32)])
def test_more_choices_than_a_block_keeps(mc, T, E, k, dtype):
    """Long calls, whose choices are not kept in shared memory until their rows are known."""
    l = logits_for(T, E, dtype, E)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9
    got = forward(mc, l.to(DEV), k, mask.to(DEV))
    chosen, slots, offsets = by_sorting(l, k, mask)
    assert torch.equal(got["experts"].cpu().long(), chosen) and torch.equal(got["slots"].cpu().long(), slots)
    assert torch.equal(got["offsets"].cpu().long(), offsets) and torch.equal(got["counts"].cpu().long(), offsets.diff())
    p = torch.softmax(l.double(), dim=1)
    want = torch.where(chosen >= 0, p.gather(1, chosen.clamp_min(0)), 0.0)
    units = p_units(l[:64].double().numpy(), chosen[:64].numpy(), False)[0].max() + 40    # (the spread of these logits, with room)
    assert ((got["gates"].cpu().double() - want).abs() <= units * U * want + 2.0 ** -126).all()
    M = int(offsets[-1])
    loss = float(E * k / M ** 2 * (offsets.diff().double() * p[mask].sum(0)).sum())
    assert abs(float(got["loss"]) - loss) <= (units + 32 + 40 + E / 32 + T / 240) * U * loss


def test_logits_past_32_bits(mc):
    """Rows whose elements lie past 2^31 of the first."""
    T, E, ld = 2100, 40, 1100000
    wide = torch.empty(T * ld, dtype=BF, device=DEV).as_strided((T, E), (ld, 1))
    l = logits_for(T, E, BF, 6)
    wide.copy_(l)
    got, want = forward(mc, wide, 3), forward(mc, l.to(DEV), 3)
    assert all(torch.equal(got[n], want[n]) for n in got)
    G, a = torch.randn(T, 3, device=DEV), torch.empty(T, E, dtype=BF, device=DEV)
    mc.route_backward(l.to(DEV), got["experts"], got["offsets"], a, dgates=G)
    mc.route_backward(wide, got["experts"], got["offsets"], wide, dgates=G)
    assert torch.equal(wide, a)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E", [(4, 6), (32, 70), (8, 300), (33, 6), (700, 70), (40, 300)])
def test_without_a_choice_a_gate_is_zero(mc, T, E, dtype, normalize):
    """Also next to gates that are NaN, in rows with fewer logits than choices."""
    l = torch.full((T, E), -INF)
    l[0, 2], l[1, 3], l[1, 1], l[2, 4] = NAN, INF, 1.0, -INF
    l[3:] = logits_for(T - 3, E, F32, 1)
    got = forward(mc, l.to(dtype).to(DEV), 4, normalize=normalize)
    want = ref.choose(l.to(dtype).double().numpy(), 4, None)
    assert np.array_equal(got["experts"].cpu().numpy(), want) and list(want[1]) == [3, 1, -1, -1] and list(want[2]) == [-1] * 4
    gates = got["gates"].cpu()
    assert not gates[torch.from_numpy(want) < 0].any()
    assert torch.isnan(gates[0, 0]) and torch.isnan(gates[1]).any() and not torch.isnan(gates[3:]).any()

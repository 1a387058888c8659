"""GPU tests of clipping at the ends of fp32's range, of lists that are clipped partly in place, and of long sums, against 64 bits.

Units are 2^-24, relative, counted from the kernels as they are.  A thread adds the squares of its 4 words of a piece (16384 bytes), 8 or
4 a word: one rounding each, the product's among them, and for values in fp32's middle range two more for the words and one for the piece.
Then 5 shuffles and 8 warps; of the partial sums 5 a round, 5 shuffles and 8 warps.  The root halves the error and has one of its own.  A
clipped value has the norm's error, the factor's two roundings, its own product's and half a step of its type; below 2^-126, where fp32 holds
multiples of 2^-149 and bf16 those of 2^-133, half such a step for each of two products and for the type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: U}
LEAST = {BF: 2.0 ** -134 + 2.0 ** -149, F32: 2.0 ** -149}
INF = float("inf")
BLOCKS, WORDS = 1216, 1024      # of a launch; of a piece


@pytest.fixture(scope="module")
def mc():
    import mlp_latency_gb300
    mlp_latency_gb300.build()
    return mlp_latency_gb300


def units(tensors):
    """Of the norm."""
    pieces = sum(max(1, -(-t.numel() * t.element_size() // (16 * WORDS))) for t in tensors)
    per = max(16 // t.element_size() for t in tensors)
    return ((4 * per + 3) * -(-pieces // BLOCKS) + 5 + 8 + 5 + 5 + 8) / 2 + 1


def clip(mc, tensors, max_norm, eps=0.0, shift=0, out_shift=None):
    """The norm, and the clipped values (in place where out_shift is None) of tensors that begin `shift` elements after a 16-byte word."""
    def placed(t, by):
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
        buf[by:].copy_(t.reshape(-1))
        return buf[by:]

    src = [placed(t, shift) for t in tensors]
    out = None if out_shift is None else [placed(torch.zeros_like(t), out_shift) for t in tensors]
    norm = torch.empty(1, device=DEV)
    ws = torch.empty(mc.clip_workspace_size(len(tensors)), dtype=torch.uint8, device=DEV)
    mc.clip_gradients(src, max_norm, norm, out=out, eps=eps, workspace=ws)
    return float(norm), src if out is None else out


def expect(tensors, got, max_norm, eps=0.0):
    """Compares a clip's result with the definition in 64 bits."""
    norm, out = got
    n = float(torch.stack([t.double().square().sum() for t in tensors]).sum().sqrt())
    max_norm, eps = float(np.float32(max_norm)), float(np.float32(eps))
    c = 1.0 if n == 0 or max_norm >= n + eps else max_norm / (n + eps)
    e = units(tensors)
    if n < 2.0 ** 128 * (1 - e * U):
        assert abs(norm - n) <= e * U * n + 2.0 ** -150, (norm, n)
    elif n > 2.0 ** 128 * (1 + e * U):
        assert norm == INF
    for t, o in zip(tensors, out):
        want = t.reshape(-1).to(DEV).double() * c
        tol = (((e + 3) * U + HALF[t.dtype]) * want.abs() * (1 + 2.0 ** -7) + LEAST[t.dtype]) if c < 1 else 0 * want
        assert bool(((o.double() - want).abs() <= tol).all()), float(((o.double() - want).abs() - tol).max())


PLACES = [dict(), dict(shift=1), dict(out_shift=0), dict(shift=3, out_shift=2)]


def normal(n, dtype, scale, seed=1):
    t = torch.randn(n, generator=torch.Generator().manual_seed(seed)).clamp(-3, 3)
    return (t.double() * scale).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [50_000, 200_000, 3_000_000])
def test_many_values_near_the_largest(mc, n, dtype):
    """The sum of their squares is past 2^270; the factor is an ordinary number."""
    t = torch.full((n,), 3e38).to(dtype)
    for place in PLACES:
        expect([t], clip(mc, [t], 1e5, **place), 1e5)


FACTORS = [(1e38, 10000, 1e-3), (1e38, 10000, 1e-6), (1e38, 10000, 1e-20), (1e38, 10000, 1e-38), (1e38, 10, 2.0 ** -149), (3e38, 200_000, 1.0),
           (1e30, 1000, 1e-20), (1e20, 1000, 1e-30), (1.0, 1000, 1e-40), (1e-10, 1000, 1e-45), (1e38, 300_000, 0.0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,n,limit", FACTORS)
def test_a_factor_below_the_least_normal_number(mc, scale, n, limit, dtype):
    """limit / norm is below 2^-126, down to 2^-297; what it leaves of a value is not."""
    t = normal(n, dtype, scale) if scale < 3e38 else torch.full((n,), scale).to(dtype)
    small = normal(77, dtype, 1e-3 * scale, 2)
    for place in PLACES:
        expect([t, small], clip(mc, [t, small], limit, **place), limit)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_large_eps(mc, dtype):
    """norm + eps is past fp32's largest value."""
    t = normal(9, dtype, 1e38)
    for place in PLACES:
        for limit in (1e38, 1.0, 3.4e38):
            expect([t], clip(mc, [t], limit, eps=3.3e38, **place), limit, eps=3.3e38)


def test_a_norm_or_a_workspace_within_the_tensors_is_refused(mc):
    size = mc.clip_workspace_size(2)
    buf = torch.zeros(size // 4 + 512, device=DEV)
    a, b, norm, ws = buf[:128], buf[128:256], buf[256:257], buf[512:]
    mc.clip_gradients([a], 1.0, norm, out=[b], workspace=ws)
    mc.gradient_norm([a, b], a[:1], workspace=ws)
    for call in (lambda: mc.clip_gradients([a, b], 1.0, b[127:], workspace=ws), lambda: mc.clip_gradients([a], 1.0, b[:1], out=[b], workspace=ws),
                 lambda: mc.clip_gradients([a], 1.0, a[7:8], out=[b], workspace=ws), lambda: mc.clip_gradients([a], 1.0, ws[5:6], workspace=ws),
                 lambda: mc.clip_gradients([a, ws[:1]], 1.0, norm, workspace=ws), lambda: mc.clip_gradients([a], 1.0, norm, out=[ws[64:192]], workspace=ws),
                 lambda: mc.gradient_norm([ws[100:228]], norm, workspace=ws)):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    torch.cuda.synchronize()
    assert not buf[:512].any()


@pytest.mark.parametrize("limit", [0.3, 5.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_some_in_place(mc, dtype, limit):
    """Lists of tensors in place, elsewhere and elsewhere in their words, in turn; the gradients of the last two stay."""
    for n in (5, 66, 1003):
        kept = [normal(1 + 977 * (i % 23), dtype, 1.0, i) for i in range(n)]
        size = sum(t.numel() for t in kept) ** 0.5
        bufs = [torch.empty(t.numel() + 1, dtype=dtype, device=DEV) for t in kept]
        src = [b[i % 2:i % 2 + t.numel()] for i, (b, t) in enumerate(zip(bufs, kept))]
        for s, t in zip(src, kept):
            s.copy_(t)
        outs = [torch.zeros(t.numel() + 1, dtype=dtype, device=DEV) for t in kept]
        out = [s if i % 3 == 0 else o[(i + i // 2) % 2:][:s.numel()] for i, (s, o) in enumerate(zip(src, outs))]
        norm = torch.empty(1, device=DEV)
        ws = torch.empty(mc.clip_workspace_size(n), dtype=torch.uint8, device=DEV)
        mc.clip_gradients(src, limit * size, norm, out=out, eps=0.0, workspace=ws)
        expect(kept, (float(norm), out), limit * size)
        for i, (s, t) in enumerate(zip(src, kept)):
            assert i % 3 == 0 or torch.equal(s.cpu(), t)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [9_000, 10_000_019, 300_000_007])
def test_long_sums_of_equal_values(mc, n, dtype):
    """Their roundings all go the same way."""
    for value in (0.1, 0.7):
        t = torch.full((n,), value, dtype=dtype, device=DEV)
        want = float(t[:1].double()) * n ** 0.5
        norm, ws = torch.empty(1, device=DEV), torch.empty(mc.clip_workspace_size(1), dtype=torch.uint8, device=DEV)
        mc.gradient_norm([t], norm, workspace=ws)
        assert abs(float(norm) - want) <= units([t]) * U * want, abs(float(norm) / want - 1) / U

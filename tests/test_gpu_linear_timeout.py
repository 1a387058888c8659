"""GPU tests of bounded waits that run out: a product whose tile takes longer than the handle's limit ends with the status TIMEOUT,
and leaves the GPU as it was for the calls after it.

The limit is 20 us.  A tile, or a slice of one, has 512 k blocks or more here, of which an SM takes in at least 18 KB each: at 64
bytes a cycle and 2.1 GHz 70 us, which the epilogue waits for.
"""
import pytest
import torch

from test_gpu_linear import BF, DEV, blank, draw, mc  # noqa: F401

pytestmark = pytest.mark.gpu
LIMIT_US = 20

# rows, K, N, counts, what is asked for
LONG = {"reduce on single CTAs": (262144, 256, 256, None, "dW"),
        "reduce on pairs": (131072, 2304, 2304, None, "dW"),
        "reduce on pairs, masked tails": (131072 + 77, 1664, 1664, [65536 + 33, 65536 + 5], "dW"),
        "rows, split": (128, 131072, 4096, None, "Y"),
        "rows, exchanged, split": (24, 524288, 512, None, "Y"),
        "rows, exchanged, on pairs": (200, 131072, 19456, None, "Y"),
        "by expert, split": (300, 131072, 512, [100, 0, 150, 50], "Y")}


@pytest.mark.parametrize("case", LONG)
def test_a_wait_that_runs_out_ends_the_launch(mc, case):  # noqa: F811
    rows, K, N, counts, what = LONG[case]
    E = len(counts or ())
    lead = (E,) if E else ()
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    X = new(rows, K)
    off = None
    if E:
        off = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(E)], dtype=torch.int32, device=DEV)
    with mc.Linear(K, N, experts=E) as patient, mc.Linear(K, N, experts=E, timeout_us=LIMIT_US) as hasty:
        plan = hasty.plan(rows, what)
        if what == "Y":
            W, out = new(*lead, K, N), [blank(rows, N, 0) for _ in range(2)]
            run = lambda lin, o: lin.forward(X, W, o, offsets=off)  # noqa: E731
        else:
            dY, out = new(rows, N), [torch.full(lead + (K, N), float("nan"), dtype=BF, device=DEV) for _ in range(2)]
            run = lambda lin, o: lin.backward(dY, X, None, dW=o, offsets=off)  # noqa: E731
        run(patient, out[0])
        assert patient.check() == 0, plan
        scrap = torch.empty_like(out[0])
        for _ in range(3):
            run(hasty, scrap)
            assert hasty.check() == mc.ERR_TIMEOUT, plan
            assert hasty.check() == 0
            run(patient, out[1])
            assert patient.check() == 0 and torch.equal(out[0], out[1]), plan


def test_both_gradients_in_one_launch_end_too(mc):  # noqa: F811
    rows, K, N = 131072, 256, 264
    X, dY, W = draw((rows, K), 1.0, 1).to(DEV), draw((rows, N), 1.0, 2).to(DEV), draw((K, N), 0.1, 3).to(DEV)
    with mc.Linear(K, N) as patient, mc.Linear(K, N, timeout_us=LIMIT_US) as hasty:
        ws = torch.empty(patient.workspace_size(rows), dtype=torch.uint8, device=DEV)
        outs = []
        for lin, status in ((patient, 0), (hasty, mc.ERR_TIMEOUT), (patient, 0)):
            dX, dW, db = blank(rows, K, 0), torch.empty_like(W), torch.empty(N, dtype=BF, device=DEV)
            lin.backward(dY, X, W, dX=dX, dW=dW, dbias=db, workspace=ws)
            assert lin.check() == status
            outs.append((dX, dW, db))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))


def test_the_calls_after_it_store_nothing_until_it_is_read(mc):  # noqa: F811
    """Also those whose launch came onto the SMs before the wait ran out: the long product here has 4 tiles, beside which the next
    launch starts at once."""
    rows, K, N = 262144, 256, 256
    X, dY, W, b = draw((rows, K), 1.0, 1).to(DEV), draw((rows, N), 1.0, 2).to(DEV), draw((K, N), 0.1, 3).to(DEV), draw((N,), 1.0, 4).to(DEV)
    few = slice(0, 512)
    dW, Y, Z, dX = torch.empty_like(W), blank(512, N, 0), blank(512, N, 0), blank(512, K, 0)
    db, db2 = (torch.full((N,), float("nan"), dtype=BF, device=DEV) for _ in range(2))
    with mc.Linear(K, N, timeout_us=LIMIT_US) as lin:
        ws = torch.empty(lin.workspace_size(512), dtype=torch.uint8, device=DEV)

        def later():
            lin.forward(X[few], W, Y, bias=b, Z=Z)
            lin.backward(dY[few], None, W, dX=dX, dbias=db, workspace=ws)
            lin.backward(dY[few], None, None, dbias=db2, workspace=ws)

        for _ in range(5):
            lin.backward(dY, X, None, dW=dW)
            later()
            later()
            assert lin.check() == mc.ERR_TIMEOUT
            for t in (Y, Z, dX, db, db2):
                assert bool(torch.isnan(t.float()).all())
        later()
        assert lin.check() == 0
    for t in (Y, Z, dX, db, db2):
        assert bool(torch.isfinite(t.float()).all())
    assert torch.equal(db, db2)


@pytest.mark.parametrize("experts", [0, 2])
def test_the_launch_before_does_not_count(mc, experts):  # noqa: F811
    """A short product behind one of a millisecond, which leaves most SMs free: its launch starts beside it and waits for its end."""
    rows, K, N, n = 262144, 256, 256, 64
    lead = (experts,) if experts else ()
    X, dY, W = draw((rows, K), 1.0, 1).to(DEV), draw((rows, N), 1.0, 2).to(DEV), draw(lead + (K, N), 0.1, 3).to(DEV)
    off = torch.tensor([0, 20, n], dtype=torch.int32, device=DEV) if experts else None
    dW, Y = torch.empty(K, N, dtype=BF, device=DEV), blank(n, N, 0)
    with mc.Linear(K, N) as slow, mc.Linear(K, N, experts=experts, timeout_us=200) as lin:
        for _ in range(5):
            slow.backward(dY, X, None, dW=dW)
            lin.forward(X[:n], W, Y, offsets=off)
            assert lin.check() == 0 and slow.check() == 0
    assert bool(torch.isfinite(Y.float()).all())

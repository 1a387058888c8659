"""GPU tests of layer norm calls among other calls: from two threads, after another call's error."""
import threading

import pytest
import torch

from test_gpu_layer_norm import BF, DEV, F32, draw, mc  # noqa: F401

pytestmark = pytest.mark.gpu


def test_two_threads_with_different_widths_of_one_kernel(mc):  # noqa: F811
    """Both widths run in the same kernels with different amounts of shared memory: neither call refuses the other's launch."""
    R, failed, results = 320, [], {}

    def work(C):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                x, dy = draw((R, C), 1, BF).to(DEV), draw((R, C), 2, BF).to(DEV)
                gamma = draw((C,), 3, BF, 0.3, 1.0).to(DEV)
                mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
                first = None
                for i in range(3000):
                    y, dx = torch.empty_like(x), torch.empty_like(x)
                    mc.layer_norm_forward(x, gamma, None, y, mean=mean, rstd=rstd)
                    mc.layer_norm_backward(dy, x, gamma, mean, rstd, dx, dx_add=dy if i & 1 else None)
                    if i == 0:
                        first = (y, dx)
                stream.synchronize()
                results[C] = torch.equal(first[0], y)
        except Exception as e:  # noqa: BLE001
            failed.append((C, repr(e)))

    threads = [threading.Thread(target=work, args=(C,)) for C in (16384, 10240)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert results == {16384: True, 10240: True}


def test_an_earlier_error_is_not_a_layer_norm_error(mc):  # noqa: F811
    R, C = 9, 264
    x, gamma, dy = draw((R, C), 1, F32).to(DEV), draw((C,), 2, F32).to(DEV), draw((R, C), 3, F32).to(DEV)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    ws = torch.empty(mc.layer_norm_workspace_size(R, C), dtype=torch.uint8, device=DEV)

    def call(spoil):
        y, dx = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
        dg, db = torch.full_like(gamma, float("nan")), torch.full_like(gamma, float("nan"))
        spoil()
        mc.layer_norm_forward(x, gamma, gamma, y, mean=mean, rstd=rstd)
        spoil()
        mc.layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db, workspace=ws)
        return y, dx, dg, db

    def no_such_device():
        with pytest.raises(mc.MlpChainError):
            mc.Linear(64, 64, device=99)

    want = call(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(want, call(no_such_device)))

"""GPU tests of layer norm calls among other calls."""
import threading

import pytest
import torch

from test_gpu_layer_norm import BF, DEV, draw, mc  # noqa: F401

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

"""GPU test of what a call keeps from other threads while it waits: a launch
blocks where its stream's queue is full, and Python's other threads run on
meanwhile."""
import threading
import time

import pytest
import torch

from test_gpu_layer_use import CALLS, _operands

pytestmark = pytest.mark.gpu
ALL = dict(CALLS, **{"rms_norm, plain": lambda z, o: z.rms_norm(o["x"], o["w"], residual=o["r"]),
                     "rms_norm_backward, plain": lambda z, o: z.rms_norm_backward(o["dy"], o["x"], o["w"], o["rstd"])})


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


@pytest.mark.parametrize("name", list(ALL))
def test_other_threads_run_while_a_launch_waits(z, name):
    o = _operands(z)
    ALL[name](z, o)
    torch.cuda.synchronize()
    done, gaps = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    ticker = threading.Thread(target=tick)
    longest = 0.0
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(1_000_000_000)  # half a second
        ticker.start()
        for _ in range(2500):  # more than a queue holds
            start = time.perf_counter()
            ALL[name](z, o)
            longest = max(longest, time.perf_counter() - start)
            if longest > 0.1:
                break
    done.set()
    ticker.join()
    torch.cuda.synchronize()
    assert longest > 0.1, "no call had to wait: the test shows nothing"
    assert max(gaps) < longest / 2

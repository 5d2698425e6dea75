"""The calls of the compiled module release Python's lock while they launch: a caller that waits for room in a full
launch queue does not stop the other threads."""
import threading
import time

import pytest
import torch

import sparse_attention_09_b200 as dsa

pytestmark = pytest.mark.gpu


def test_a_full_launch_queue_stops_one_thread_only():
    x, w = torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    pos, freqs = torch.zeros(4, dtype=torch.int32, device="cuda"), dsa.dsa_rope_frequencies(64, 1e4)[0].cuda()
    dsa.dsa_rmsnorm(x, w, 1e-6, y=y)
    dsa.dsa_rope(x.view(4, 1, 64), pos, freqs, y.view(4, 1, 64), 0, 64)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():  # the longest time without a turn
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    ticker = threading.Thread(target=tick)
    ticker.start()
    time.sleep(0.02)
    begin.record()
    torch.cuda._sleep(2 * 10 ** 9)  # about a second, then the queue behind it
    end.record()
    longest = 0.0
    for _ in range(3000):  # more than the queue holds
        at = time.perf_counter()
        dsa.dsa_rmsnorm(x, w, 1e-6, y=y)
        dsa.dsa_rope(x.view(4, 1, 64), pos, freqs, y.view(4, 1, 64), 0, 64)
        longest = max(longest, time.perf_counter() - at)
    torch.cuda.synchronize()
    stop.set()
    ticker.join()
    slept = begin.elapsed_time(end) / 1000
    assert longest > slept / 2, "the launches never waited for the queue"
    assert max(gaps) < longest / 4, f"no turn for {max(gaps):.3f} s while a launch waited {longest:.3f} s"

"""Calls from several threads: one that waits for the device holds up no other."""
import threading
import time

import pytest
import torch

import mla_latent_kv_22_b200 as M

pytestmark = pytest.mark.gpu


def test_a_thread_that_reads_the_error_word_does_not_hold_up_another():
    # The waiting thread's stream is busy for over a second; the other thread's call goes
    # to a stream of its own, and the main thread needs neither.
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c_kv, k_rope, kv = torch.zeros(1, 512, **bf), torch.zeros(1, 64, **bf), torch.zeros(1, 64, 576, **bf)
    table, lens, cos_sin = torch.zeros(1, 1, **i32), torch.ones(1, **i32), torch.zeros(4, 64, device="cuda")
    append = lambda: M.mla_append(c_kv, k_rope, kv, table, lens, cos_sin)
    busy, own = torch.cuda.Stream(), torch.cuda.Stream()
    append()
    torch.cuda._sleep(1000)
    assert M.mla_get_device_error() == 0
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(3_000_000_000)   # clock cycles: a second and a half at 2 GHz
    done = torch.cuda.Event()
    done.record(busy)
    status, launched = [], []

    def wait():
        status.append(M.mla_get_device_error(busy))

    def launch():
        with torch.cuda.stream(own):
            append()
        launched.append(done.query())

    waiter, other = threading.Thread(target=wait), threading.Thread(target=launch)
    waiter.start()
    time.sleep(0.05)
    other.start()
    gap, last = 0.0, time.perf_counter()
    for _ in range(15):
        time.sleep(0.01)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    busy_until_now = not done.query()
    other.join()
    waiter.join()
    assert gap < 0.5, f"the main thread stood still for {gap:.2f} s"
    assert busy_until_now, "the busy stream ended too early to show anything"
    assert status == [0]
    assert launched == [False], "the call waited for the other thread's stream"

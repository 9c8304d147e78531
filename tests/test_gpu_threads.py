"""The calls around the layer from several threads: a call that waits on the host, since its stream's queue
of launches is full, leaves the other threads running."""

import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_waiting_launch_leaves_other_threads_running():
    from int4_quantised_moe_b200 import binding as B
    x = torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((1, 8), device="cuda")
    cfg = B.make_select_cfg(8, 2)
    ck = B.ckpt8_save(x)
    _, _, rstd, _ = B.norm_fwd(x, w)
    ids, _ = B.router_select(z, cfg)
    gr = torch.zeros((1, 2), device="cuda")
    calls = {"router_select": lambda: B.router_select(z, cfg), "router_select_bwd": lambda: B.router_select_bwd(z, cfg, ids, gr),
             "ckpt8_save": lambda: B.ckpt8_save(x), "ckpt8_load": lambda: B.ckpt8_load(ck),
             "norm_fwd": lambda: B.norm_fwd(x, w), "norm_bwd": lambda: B.norm_bwd(x, x, rstd, w)}
    # cycles of half a second or more on a clock of at most 2 GHz
    cycles = 1_000_000_000
    for name, call in calls.items():
        call()
        torch.cuda.synchronize()
        gaps, done = [], threading.Event()

        def watch():
            last = time.perf_counter()
            while not done.is_set():
                time.sleep(0.001)
                now = time.perf_counter()
                gaps.append(now - last)
                last = now

        thread = threading.Thread(target=watch)
        thread.start()
        try:
            torch.cuda._sleep(cycles)
            longest = 0.0  # of one call: the one that finds the queue full
            for _ in range(5000):
                t = time.perf_counter()
                call()
                longest = max(longest, time.perf_counter() - t)
        finally:
            done.set()
            thread.join()
            torch.cuda.synchronize()
        assert longest > 0.2, (name, longest)  # the queue was full, else this shows nothing
        assert max(gaps) < longest / 2, (name, max(gaps), longest)

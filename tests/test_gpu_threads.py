"""Calls of different sizes from several threads at once, each on a stream of its own."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def together(jobs):
    """Every job in a thread of its own; the first exception is raised here."""
    failed = []

    def body(job):
        try:
            job()
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)
    threads = [threading.Thread(target=body, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


def test_page_maps_of_large_batches():
    """Batches whose maps need 60 to 196 KB of shared memory."""
    dev = device()

    def job(batch):
        def run():
            with torch.cuda.stream(torch.cuda.Stream()):
                z = torch.zeros(batch, dtype=torch.int32, device=dev)
                table = torch.zeros((batch, 1), dtype=torch.int32, device=dev)
                free = torch.arange(4, dtype=torch.int32, device=dev)
                count = torch.tensor([4], dtype=torch.int32, device=dev)
                new = z.clone()
                new[batch - 1] = 3
                for _ in range(3000):
                    r = d2f.page_map(new, z, table, free, count, block_size=16, capacity=8,
                                     max_append=1)
                assert r["slot"].tolist() == [48, 49, 50] + [-1] * 5 and int(r["n_append"]) == 1
        return run
    together([job(b) for b in (16384, 5000, 9000, 12000)])


def test_attention_and_log_probabilities():
    """Short and long, small and large calls of the two operators with a workspace, one each."""
    from test_gpu_workspaces import attention_call, logprobs_call, workspace
    from test_gpu_kv4_attention import problem
    dev = device()
    bf, f32 = torch.bfloat16, torch.float32
    calls = [attention_call(problem(ctx, blocks, hq=h, hkv=h, D=D, B=B, dtype=dt, seed=h), dev)
             for ctx, blocks, h, D, B, dt in (
                 ([1900], [1], 4, 128, 16, bf), ([40] * 300, [1] * 300, 1, 128, 16, bf),
                 ([300, 700], [2, 1], 6, 64, 8, bf), ([500], [1], 4, 128, 16, f32))]
    calls += [logprobs_call(n, 60000, dt, 5, dev) for n, dt in ((3, bf), (300, f32))]
    torch.cuda.synchronize()

    def job(call, size):
        def body():
            with torch.cuda.stream(torch.cuda.Stream()):
                ws = workspace(size, dev)
                first = [x.clone() for x in call(ws)]
                for _ in range(300):
                    got = call(ws)
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(first, got))
        return body
    together([job(*c) for c in calls])


WINDOW_STEPS = """
import sys, threading, torch
sys.path.insert(0, %r)
from block_causal_kv_gb300 import d2f
d2f.load()
dev = torch.device("cuda:0")
caps = [38000, 12000, 20000, 30000, 36000, 15000, 25000, 11000]
start, failed = threading.Barrier(len(caps)), []
def job(cap):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            st = d2f.WindowState(dev, batch=1, block_size=1, max_blocks=4, max_pages_per_seq=4,
                                 num_free=4, mask_id=9, capacity=cap)
            torch.cuda.current_stream().synchronize()
            start.wait()
            for _ in range(20):
                d2f.window_step(st, tau_add=0.5, tau_act=1.0, use_stopped=False)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        failed.append(repr(e))
threads = [threading.Thread(target=job, args=(c,)) for c in caps]
[t.start() for t in threads]
[t.join() for t in threads]
sys.exit("; ".join(failed) if failed else 0)
"""


def test_first_window_steps_of_a_process():
    """States of 65 to 226 KB, whose first calls of a process meet (in three processes)."""
    device()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", WINDOW_STEPS % root], capture_output=True,
                           text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-500:]

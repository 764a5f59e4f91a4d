"""Calls of different sizes from several threads at once, each on a stream of its own."""
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

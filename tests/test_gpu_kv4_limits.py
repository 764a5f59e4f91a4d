"""d2f_block_attn_kv4 at the largest batch, whose per-sequence arrays fill a CTA's shared memory."""
import numpy as np
import pytest
import torch

from gpu_common import device
from test_gpu_kv4_attention import check, problem, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,B", [(128, 8), (64, 16)])
@pytest.mark.parametrize("batch", [1023, 1024])
def test_largest_batches(batch, D, B):
    """Every third sequence without a window, contexts of none to three pages."""
    dev = device()
    g = np.random.default_rng(batch + D)
    ctx = g.integers(0, 3 * B + 1, batch).tolist()
    blocks = [0 if b % 3 == 1 else 1 for b in range(batch)]
    p = problem(ctx, blocks, hq=1, hkv=1, D=D, B=B, dtype=torch.bfloat16, seed=batch)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(p, out, lse)


@pytest.mark.parametrize("cycles", [1, 300, 3000])
def test_wait_budget_runs_out_in_windows_of_several_tiles(cycles, monkeypatch):
    """Waits that give up between a window's key tiles, sooner or later in the call: it returns,
    reports them if there were any, and with a fresh workspace the next call is right."""
    dev = device()
    p = problem([100, 0, 900], [20, 9, 17], hq=2, hkv=1, D=128, B=16, dtype=torch.bfloat16, seed=5)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    monkeypatch.setenv("D2F_WAIT_CYCLES", str(cycles))
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) in (0, 5) and (cycles > 1 or int(err) == 5)
    if int(err) == 0:
        check(p, out, lse)
    monkeypatch.delenv("D2F_WAIT_CYCLES")
    err.zero_()
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(p, out, lse)

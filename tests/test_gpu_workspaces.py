"""One workspace that serves calls of different sizes, one after another: the results are those
of a fresh workspace, bit by bit."""
import numpy as np
import pytest
import torch

from gpu_common import device
from test_gpu_kv4_attention import problem

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def attention_call(p, dev):
    """A call of `problem`'s inputs as a function of the workspace, and its workspace's bytes."""
    t = [p[k].to(dev) for k in ("q", "k_win", "v_win", "pool")]
    t += [torch.from_numpy(p["table"]).to(dev), torch.tensor(p["ctx"], dtype=torch.int32, device=dev),
          torch.from_numpy(p["q_start"]).to(dev)]
    max_q = int(np.diff(p["q_start"]).max())
    dt = d2f.BF16 if p["dtype"] == torch.bfloat16 else d2f.F32
    size = d2f.attn_kv4_workspace_size(len(p["ctx"]), t[0].shape[0], max_q, max(p["ctx"]),
                                       t[0].shape[1], t[1].shape[1], p["D"], p["B"], dt)
    out = torch.empty_like(t[0])
    lse = torch.empty(t[0].shape[:2], device=dev)

    def call(ws):
        out.fill_(7)
        lse.fill_(7)
        d2f.block_attn_kv4(*t, block_size=p["B"], max_q_per_seq=max_q, max_ctx=max(p["ctx"]),
                           softmax_scale=p["scale"], out=out, lse=lse, workspace=ws)
        return out, lse
    return call, size


def workspace(size, dev):
    return torch.zeros(size, dtype=torch.uint8, device=dev)


def check_sequence(calls, order, dev):
    """The calls in this order over one workspace, then from graphs captured over it."""
    fresh = []
    for call, size in calls:
        fresh.append([x.clone() for x in call(workspace(size, dev))])
    ws = workspace(max(size for _, size in calls), dev)
    for i in order:
        got = calls[i][0](ws)
        torch.cuda.synchronize()
        for a, b in zip(got, fresh[i]):
            assert torch.equal(a, b), "call %d" % i
    graphs = []
    for call, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call(ws)
        graphs.append((g, got))
    for i in order:
        graphs[i][0].replay()
        torch.cuda.synchronize()
        for a, b in zip(graphs[i][1], fresh[i]):
            assert torch.equal(a, b), "replay %d" % i


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtypes", [(BF, BF, BF), (F32, F32, F32), (BF, F32, BF), (F32, BF, F32)],
                         ids=lambda d: "-".join(str(x)[6:] for x in d))
def test_attention_over_the_4_bit_cache(dtypes):
    """One long context, then a batch whose row tiles are cut too, then windows of more rows."""
    dev = device()
    kw = dict(D=128, B=16)
    ps = [problem([2100], [1], hq=4, hkv=4, dtype=dtypes[0], seed=1, **kw),
          problem([700, 333, 900, 64, 1200, 0, 150, 513], [1, 2, 1, 3, 1, 2, 1, 2], hq=16, hkv=16,
                  dtype=dtypes[1], seed=2, **kw),
          problem([800, 90], [9, 5], hq=14, hkv=2, dtype=dtypes[2], seed=3, **kw)]
    check_sequence([attention_call(p, dev) for p in ps], [0, 1, 2, 0, 2, 1, 0, 1], dev)

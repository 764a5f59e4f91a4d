"""One workspace that serves calls of different sizes, one after another: the results are those
of a fresh workspace, bit by bit."""
import numpy as np
import pytest
import torch

from gpu_common import device
from test_gpu_kv4_attention import problem

from block_causal_kv_gb300 import d2f, synth

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


def logprobs_call(rows, V, dtype, top_k, dev):
    g = torch.Generator(device=dev).manual_seed(rows + V)
    x = (torch.randn((rows, V), generator=g, device=dev) * 3).to(dtype)
    tok = torch.randint(0, V, (rows,), generator=g, device=dev).int()
    f, i = dict(device=dev), dict(device=dev, dtype=torch.int32)
    out = dict(logprob=torch.empty(rows, **f), entropy=torch.empty(rows, **f),
               top_id=torch.empty((rows, top_k), **i), top_logprob=torch.empty((rows, top_k), **f))

    def call(ws):
        for t in out.values():
            t.fill_(7)
        d2f.token_logprobs(x, tok, top_k=top_k, workspace=ws, **out)
        return list(out.values())
    dt = d2f.BF16 if dtype == torch.bfloat16 else d2f.F32
    return call, max(1, d2f.logprobs_workspace_size(rows, V, top_k, dt))


@pytest.mark.parametrize("top_k", [0, 5])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_log_probabilities(dtype, top_k):
    """Few rows in many slices, more rows in fewer, one row, and rows of one slice each."""
    dev = device()
    calls = [logprobs_call(n, v, dtype, top_k, dev)
             for n, v in ((48, 126464), (384, 60000), (1, 152064), (608, 40000), (700, 20000))]
    check_sequence(calls, [0, 1, 3, 2, 1, 4, 0, 3, 1, 2, 0], dev)


def test_attention_and_log_probabilities_in_turn():
    dev = device()
    p = problem([700, 333, 900, 64, 1200, 0, 150, 513], [1, 2, 1, 3, 1, 2, 1, 2], hq=4, hkv=4, D=64,
                B=16, dtype=BF, seed=5)
    calls = [attention_call(p, dev), attention_call(dict(p, dtype=F32, **{
        k: p[k].float() for k in ("q", "k_win", "v_win")}), dev)]
    calls += [logprobs_call(n, 60000, BF, 9, dev) for n in (20, 400)]
    check_sequence(calls, [0, 3, 1, 2, 0, 2, 3, 1, 0], dev)


@pytest.mark.parametrize("form", ["float32", "stream-k"])
def test_attention_over_the_unquantised_cache(form, monkeypatch):
    dev = device()
    if form == "stream-k":
        for k in ("D2F_ATTN_SK", "D2F_TC_DEEP"):
            monkeypatch.setenv(k, "1")
        monkeypatch.setenv("D2F_TC_ROWS", "128")
    dt = F32 if form == "float32" else BF
    calls = []
    for batch, heads, seed in ((1, 2, 1), (6, 16, 2), (2, 3, 3)):
        w = synth.Workload("turn%d" % seed, batch, heads, heads, 128, 16, dt, [1500 // batch] * batch,
                           [2] * batch, 64, permute_pages=True, seed=seed)
        p = synth.make_problem(w)
        g = p.to(dev)
        kw = dict(block_size=16, max_q_per_seq=p.max_q_per_seq, max_ctx=p.max_ctx)
        size = d2f.attn_workspace_size(batch, w.total_q, p.max_q_per_seq, p.max_ctx, heads, heads,
                                       128, 16, d2f.F32 if dt == F32 else d2f.BF16)
        out, lse = torch.empty_like(g.q), torch.empty(g.q.shape[:2], device=dev)

        def call(ws, g=g, out=out, lse=lse, kw=kw):
            out.fill_(7)
            lse.fill_(7)
            d2f.block_attn(g.q, g.k_win, g.v_win, g.k_pool, g.v_pool, g.page_table, g.ctx_len,
                           g.q_start, out=out, lse=lse, workspace=ws, **kw)
            return out, lse
        calls.append((call, size))
    check_sequence(calls, [0, 1, 2, 0, 2, 1, 0, 1], dev)

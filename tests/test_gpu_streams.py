"""Calls on a stream of their own (`stream=`) that make their results and workspace themselves:
nothing of them waits for, or is overwritten by, work on the stream that is current."""
import numpy as np
import pytest
import torch

from gpu_common import device
from test_gpu_kv4_attention import problem

from block_causal_kv_gb300 import d2f, synth

pytestmark = pytest.mark.gpu

PAUSE = 100_000_000  # cycles (some 50 ms) that the current stream is kept busy
NAMES = ["attention bf16", "attention f32", "log probabilities", "read", "page map",
         "block attention f32", "commit"]


def make(name, dev):
    """(call(stream) -> the tensors it made, bytes of its workspace)."""
    if name.startswith("attention"):
        dt = torch.bfloat16 if name.endswith("bf16") else torch.float32
        p = problem([2100, 700], [1, 2], hq=8, hkv=8, D=128, B=16, dtype=dt, seed=1)
        t = [p[k].to(dev) for k in ("q", "k_win", "v_win", "pool")]
        t += [torch.from_numpy(p["table"]).to(dev),
              torch.tensor(p["ctx"], dtype=torch.int32, device=dev),
              torch.from_numpy(p["q_start"]).to(dev)]
        size = d2f.attn_kv4_workspace_size(2, 48, 32, 2100, 8, 8, 128, 16,
                                           d2f.BF16 if dt == torch.bfloat16 else d2f.F32)
        return lambda s: d2f.block_attn_kv4(*t, block_size=16, max_q_per_seq=32, max_ctx=2100,
                                            stream=s), size
    g = torch.Generator(device=dev).manual_seed(2)
    if name == "log probabilities":
        x = torch.randn((40, 126464), generator=g, device=dev).bfloat16()
        tok = torch.randint(0, 126464, (40,), generator=g, device=dev).int()
        size = d2f.logprobs_workspace_size(40, 126464, 6)
        return lambda s: list(d2f.token_logprobs(x, tok, top_k=6, stream=s).values()), size
    if name == "read":
        pool = torch.randint(0, 127, (64, 4, 2304), generator=g, device=dev, dtype=torch.uint8)
        slot = torch.randperm(1024, generator=g, device=dev)
        return lambda s: d2f.kv4_read(pool, slot, head_dim=128, block_size=16, stream=s), 0
    if name == "page map":
        new = torch.randint(0, 900, (50,), generator=g, device=dev).int()
        ctx = torch.zeros(50, dtype=torch.int32, device=dev)
        free = torch.randperm(4000, generator=g, device=dev).int()
        count = torch.tensor([4000], dtype=torch.int32, device=dev)
        table = torch.full((50, 60), -1, dtype=torch.int32, device=dev)

        def call(s):
            r = d2f.page_map(new, ctx, table, free, count, block_size=16, capacity=50000,
                             max_append=4000, stream=s)
            return [r[k] for k in sorted(r) if k != "page_table"]
        return call, 0
    if name == "commit":
        p = synth.make_problem(synth.small("llada"))
        q = p.to(dev)
        size = d2f.commit_workspace_size(p.w.total_q, p.w.vocab, p.w.block_size)

        state = [(q.tokens.clone(), q.masked.clone()) for _ in range(4)]  # one a call

        def call(s):
            r = d2f.commit(q.logits, *state.pop(), q.q_start, q.block_phase, q.tau,
                           block_size=p.w.block_size, mask_id=p.mask_id, stream=s)
            return [r[k] for k in ("conf", "argmax", "block_remaining")]
        return call, size
    w = synth.Workload("side", 2, 4, 4, 64, 16, torch.float32, [700, 300], [2, 1], 64, seed=4)
    p = synth.make_problem(w)
    q = p.to(dev)
    size = d2f.attn_workspace_size(2, w.total_q, p.max_q_per_seq, p.max_ctx, 4, 4, 64, 16, d2f.F32)
    return lambda s: d2f.block_attn(q.q, q.k_win, q.v_win, q.k_pool, q.v_pool, q.page_table,
                                    q.ctx_len, q.q_start, block_size=16,
                                    max_q_per_seq=p.max_q_per_seq, max_ctx=p.max_ctx,
                                    stream=s), size


def expected(call):
    """The results of a call on the current stream, whose own memory keeps nothing of them."""
    got = call(None)
    want = [x.clone() for x in got]
    for x in got:
        x.fill_(3)
    torch.cuda.synchronize()
    return want


def same(a, b):
    return all(torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(a, b))


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("read", "page map")])
def test_workspace_made_behind_a_busy_current_stream(name, monkeypatch):
    """The workspace's zeros are part of the call's stream, not of the busy one."""
    dev = device()
    call, size = make(name, dev)
    want = expected(call)
    side = torch.cuda.Stream()
    old = torch.full((size,), 0x7f, dtype=torch.uint8, device=dev)  # the workspace's memory
    torch.cuda.synchronize()
    real = torch.zeros
    monkeypatch.setattr(torch, "zeros",
                        lambda n, **kw: old.zero_() if n == size else real(n, **kw))
    torch.cuda._sleep(PAUSE)
    got = call(side)
    side.synchronize()
    busy = not torch.cuda.current_stream().query()
    with torch.cuda.stream(side):
        got = [x.clone() for x in got]
    torch.cuda.synchronize()
    assert busy, "the pause was too short to show anything"
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_results_share_no_memory_with_pending_work(name):
    """Memory freed on the current stream, with work on it still queued there, does not become
    the results of a call on another stream."""
    dev = device()
    call, _ = make(name, dev)
    want = expected(call)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty_like(x) for x in want for _ in range(16)]
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    for x in held:
        x.fill_(3)
    del x, held
    got = call(side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_results_stay_the_callers_until_it_is_done(name):
    """Results dropped while the current stream still reads them are not handed out again on the
    call's stream before that."""
    dev = device()
    call, _ = make(name, dev)
    want = expected(call)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    kept = [x.clone() for x in got]
    shapes = [(x.shape, x.dtype) for x in got]
    del got
    with torch.cuda.stream(side):
        other = [torch.full(s, 3, dtype=t, device=dev) for s, t in shapes]
    torch.cuda.synchronize()
    assert same(kept, want) and len(other) == len(kept)


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_forked_stream(name):
    """A captured call on a stream that was forked off the capturing one."""
    dev = device()
    call, _ = make(name, dev)
    want = expected(call)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(1 if name == "commit" else 3):  # (a commit changes its state)
        for x in got:
            x.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want)


def test_results_without_elements():
    """No alternatives, no rows, no list: tensors without memory, made on another stream."""
    dev = device()
    side = torch.cuda.Stream()
    x = torch.randn((2, 50), device=dev)
    tok = torch.tensor([3, 4], dtype=torch.int32, device=dev)
    zero, none = tok[:0], torch.zeros((0, 3), dtype=torch.int32, device=dev)
    count = torch.tensor([1], dtype=torch.int32, device=dev)
    pool = d2f.kv4_pool(dev, num_pages=1, num_heads_kv=1, head_dim=64, block_size=8)
    torch.cuda.synchronize()
    r = d2f.token_logprobs(x, tok, top_k=0, stream=side)
    m = d2f.page_map(zero, zero, none, tok, count, block_size=8, capacity=0, max_append=0, stream=side)
    k, v = d2f.kv4_read(pool, torch.zeros(0, dtype=torch.int64, device=dev), head_dim=64,
                        block_size=8, stream=side)
    torch.cuda.synchronize()
    want = torch.log_softmax(x.double(), -1)[[0, 1], tok.long()]
    assert torch.allclose(r["logprob"].double(), want, atol=1e-5) and r["top_id"].shape == (2, 0)
    assert m["slot"].numel() == 0 and m["row_start"].tolist() == [0] and int(m["free_count"]) == 1
    assert k.shape == v.shape == (0, 1, 64)

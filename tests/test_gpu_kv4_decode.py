"""The 4-bit cache's operators together, as a decode uses them: prompts laid out by the page
map and quantised into its pages, then one captured graph per step (append of the finished
blocks, attention, commit, log probabilities of the candidates, window scheduler) against a
host loop over the plain forms and the oracle's commit and scheduler."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import oracle
from gpu_common import device
from test_gpu_logprobs import check as check_logprobs
from test_gpu_window import _compare, _host

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu

K_EXP, V_EXP = 1, -2


def store(pool, k, v, src, dst, rows, B):
    """The listed rows' bytes into a host pool, and nothing else."""
    for s, p, n in zip(src, dst, rows):
        for h in range(k.shape[1]):
            x = np.zeros((2, B, k.shape[2]))
            x[0, :n], x[1, :n] = k[s:s + n, h].double(), v[s:s + n, h].double()
            kc, kb, _ = ref.encode(x[0], K_EXP)
            vc, vb, _ = ref.encode(x[1], V_EXP)
            pool[p, h] = ref.page_tile(kc, kb, vc, vb)


def values(pool, B, D):
    kv = np.zeros(pool.shape[:2] + (B, D))
    vv = np.zeros_like(kv)
    for p in range(pool.shape[0]):
        for h in range(pool.shape[1]):
            kv[p, h], vv[p, h] = ref.tile_values(pool[p, h], B, D, K_EXP, V_EXP)
    return kv, vv


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_from_prompts_to_the_last_block(dtype):
    dev = device()
    batch, B, W, Hq, Hkv, D, V, TOP = 4, 16, 3, 4, 2, 128, 200, 5
    prompt, gen = [0, 16, 160, 48], [3, 2, 4, 1]
    mask_id, tau_add, tau_act = V, 0.25, 0.75
    g = torch.Generator().manual_seed(17)
    pages = sum(prompt) // B + sum(gen) + 3
    st = d2f.WindowState(dev, batch=batch, block_size=B, max_blocks=W, max_pages_per_seq=16,
                         num_free=pages, mask_id=mask_id)
    st.stopped = None
    st.gen_blocks.copy_(torch.tensor(gen, dtype=torch.int32))
    st.free_pages.copy_(torch.randperm(pages, generator=g).to(torch.int32))
    st.free_count.fill_(pages)
    cap = st.capacity
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    pool = d2f.kv4_pool(dev, num_pages=pages, num_heads_kv=Hkv, head_dim=D, block_size=B)
    host_pool = np.zeros(tuple(pool.shape), np.uint8)

    # ---- prompts: pages, then their K/V, without a readback -----------------------------
    def draw(n, h):
        return torch.randn((n, h, D), generator=g).to(dtype)
    rows = sum(prompt)
    pk, pv = draw(rows, Hkv), draw(rows, Hkv)
    m = d2f.page_map(torch.tensor(prompt, dtype=torch.int32, device=dev), st.ctx_len, st.page_table,
                     st.free_pages, st.free_count, block_size=B, capacity=rows + 5,
                     max_append=pages, ctx_len_out=st.ctx_len, free_count_out=st.free_count, err=err)
    d2f.kv4_append(pk.to(dev), pv.to(dev), m["app_src"], m["app_dst"], pool, block_size=B,
                   n_rows=m["app_rows"], k_exp=K_EXP, v_exp=V_EXP, n_append_dev=m["n_append"],
                   err=err)
    n = int(m["n_append"])
    assert int(err) == 0 and n == rows // B and st.ctx_len.tolist() == prompt
    store(host_pool, pk, pv, m["app_src"][:n].tolist(), m["app_dst"][:n].tolist(), [B] * n, B)
    assert np.array_equal(pool.cpu().numpy(), host_pool)
    k, v = d2f.kv4_read(pool, m["slot"], head_dim=D, block_size=B, dtype=dtype, k_exp=K_EXP,
                        v_exp=V_EXP, err=err)
    assert np.array_equal(k[:rows].double().cpu().numpy(), ref.encode(pk.double().numpy(), K_EXP)[2])
    assert np.array_equal(v[:rows].double().cpu().numpy(), ref.encode(pv.double().numpy(), V_EXP)[2])
    assert not k[rows:].any() and not v[rows:].any()

    # ---- the step ------------------------------------------------------------------------
    # (logits as in the oracle loop test: confident or flat rows, far from tau)
    q, kw, vw = draw(cap, Hq), draw(cap, Hkv), draw(cap, Hkv)
    logits = torch.zeros(cap, V)
    sure = torch.rand(cap, generator=g) < 0.35
    peak = torch.randint(0, V, (cap,), generator=g)
    logits[sure] = -100.0
    logits[sure, peak[sure]] = 0.0
    logits = logits.to(dtype)
    d = {name: t.to(dev) for name, t in dict(q=q, kw=kw, vw=vw, logits=logits).items()}
    tau = torch.full((batch,), 0.5, device=dev)
    max_ctx = max(p + x * B for p, x in zip(prompt, gen))
    code = d2f.BF16 if dtype == torch.bfloat16 else d2f.F32
    out, lse = torch.empty_like(d["q"]), torch.empty((cap, Hq), device=dev)
    amax = torch.full((cap,), -1, dtype=torch.int32, device=dev)
    ws_a = d2f.attn_kv4_workspace(dev, batch=batch, total_q=cap, max_q_per_seq=W * B,
                                  max_ctx=max_ctx, num_heads_q=Hq, num_heads_kv=Hkv, head_dim=D,
                                  block_size=B, dtype=code)
    ws_c = d2f.commit_workspace(dev, total_q=cap, vocab=V, block_size=B, dtype=code)
    ws_l = d2f.logprobs_workspace(dev, n=cap, vocab=V, top_k=TOP, dtype=code)
    lp = dict(logprob=torch.empty(cap, device=dev), entropy=torch.empty(cap, device=dev),
              top_id=torch.empty((cap, TOP), dtype=torch.int32, device=dev),
              top_logprob=torch.empty((cap, TOP), device=dev))

    def step():
        d2f.kv4_append(d["kw"], d["vw"], st.app_src, st.app_dst, pool, block_size=B, k_exp=K_EXP,
                       v_exp=V_EXP, n_append_dev=st.n_append, err=err)
        d2f.block_attn_kv4(d["q"], d["kw"], d["vw"], pool, st.page_table, st.ctx_len, st.q_start,
                           block_size=B, max_q_per_seq=W * B, max_ctx=max_ctx, k_exp=K_EXP,
                           v_exp=V_EXP, out=out, lse=lse, workspace=ws_a, err=err)
        d2f.commit(d["logits"], st.tokens, st.masked, st.q_start, st.block_phase, tau,
                   block_size=B, mask_id=mask_id, argmax=amax, workspace=ws_c, err=err)
        d2f.token_logprobs(d["logits"], amax, top_k=TOP, workspace=ws_l, err=err, **lp)
        d2f.window_step(st, tau_add=tau_add, tau_act=tau_act, err=err, use_stopped=False)

    want = _host(st)
    want = oracle.window_step(want, B, W, mask_id, tau_add, tau_act)
    stream = torch.cuda.Stream(device=dev)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        d2f.window_step(st, tau_add=tau_add, tau_act=tau_act, err=err, use_stopped=False)
        stream.synchronize()
        _compare(st, want, err, "first window")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    looked = 0
    for i in range(100):
        live = int(want["q_start"][-1])
        if live == 0:
            break
        graph.replay()
        stream.synchronize()
        assert int(err) == 0, "step %d: device error %d" % (i, int(err))
        if want["n_append"]:
            src, dst = want["app_src"].tolist(), want["app_dst"].tolist()
            store(host_pool, kw, vw, src, dst, [B] * len(src), B)
        assert np.array_equal(pool.cpu().numpy(), host_pool), "step %d: pages" % i
        c = oracle.commit(logits[:live], want["tokens"][:live], want["masked"][:live],
                          want["q_start"], want["block_phase"][:live // B], tau.cpu(), B, mask_id)
        if i % 3 == 0:
            looked += 1
            kv, vv = values(host_pool, B, D)
            ctx, qs = want["ctx_len"].tolist(), want["q_start"].tolist()
            o, l, ac, aw, sabs = ref.attention(q, kw, vw, kv, vv, want["page_table"].numpy(), ctx,
                                               qs, B, D ** -0.5)
            bo, bl = ref.attention_bounds(o, ac, aw, sabs, D, max(ctx) + W * B,
                                          dtype == torch.bfloat16)
            assert (np.abs(out.double().cpu().numpy() - o)[:live] <= bo[:live]).all()
            assert (np.abs(lse.double().cpu().numpy() - l)[:live] <= bl[:live]).all()
            tok = torch.where(want["masked"] != 0, logits.float().argmax(-1).to(torch.int32),
                              torch.tensor(-1, dtype=torch.int32))
            # (the commit leaves the rows past q_start[batch] as they are)
            assert torch.equal(amax[:live].cpu(), tok[:live])
            check_logprobs(logits[:live], tok[:live].tolist(), TOP,
                           {name: t[:live] for name, t in lp.items()})
        tok, msk = want["tokens"].clone(), want["masked"].clone()
        tok[:live], msk[:live] = c["tokens"], c["masked"]
        want = oracle.window_step(dict(want, tokens=tok, masked=msk, stopped=None), B, W, mask_id,
                                  tau_add, tau_act)
        _compare(st, want, err, "step %d" % i)
    else:
        raise AssertionError("decode did not finish")
    assert looked >= 2
    assert st.ctx_len.tolist() == [p + x * B for p, x in zip(prompt, gen)]


def test_an_append_behind_a_refused_page_map_writes_nothing():
    dev = device()
    pool = torch.full((4, 2, 2304), 0xA5, dtype=torch.uint8, device=dev)
    x = torch.randn((64, 2, 128), device=dev).to(torch.bfloat16)
    for capacity in (32, 300000):
        i32 = dict(dtype=torch.int32, device=dev)
        err = torch.zeros(1, **i32)
        m = d2f.page_map(torch.tensor([20, -1], **i32), torch.zeros(2, **i32),
                         torch.full((2, 4), -1, **i32), torch.arange(4, **i32),
                         torch.tensor([4], **i32), block_size=16, capacity=capacity, max_append=4,
                         err=err)
        # (whatever the list's memory holds)
        m["app_src"].zero_()
        m["app_dst"].copy_(torch.arange(4, **i32))
        d2f.kv4_append(x, x, m["app_src"], m["app_dst"], pool, block_size=16,
                       n_append_dev=m["n_append"])
        assert int(err) == 1 and int(m["n_append"]) == -1 and (pool == 0xA5).all()


def test_two_calls_at_once_with_a_workspace_each():
    """Two layers' attention and log probabilities on two streams, interleaved."""
    from test_gpu_kv4_attention import problem
    dev = device()
    jobs = []
    for seed in (5, 6):
        p = problem([3000, 64, 700], [2, 1, 3], hq=8, hkv=4, D=128, B=16, dtype=torch.bfloat16,
                    seed=seed)
        n = np.diff(p["q_start"])
        t = [p[k].to(dev) for k in ("q", "k_win", "v_win", "pool")] + [
            torch.from_numpy(p["table"]).to(dev),
            torch.tensor(p["ctx"], dtype=torch.int32, device=dev),
            torch.from_numpy(p["q_start"]).to(dev)]
        x = torch.randn((40, 30000), generator=torch.Generator().manual_seed(seed)).to(dev)
        tok = torch.arange(40, dtype=torch.int32, device=dev)
        ws = d2f.attn_kv4_workspace(dev, batch=3, total_q=t[0].shape[0], max_q_per_seq=int(n.max()),
                                    max_ctx=3000, num_heads_q=8, num_heads_kv=4, head_dim=128,
                                    block_size=16)
        wl = d2f.logprobs_workspace(dev, n=40, vocab=30000, top_k=3, dtype=d2f.F32)
        jobs.append((t, dict(block_size=16, max_q_per_seq=int(n.max()), max_ctx=3000, workspace=ws),
                     x, tok, wl))

    def once(job, stream=None):
        t, kw, x, tok, wl = job
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            o, l = d2f.block_attn_kv4(*t, **kw)
            r = d2f.token_logprobs(x, tok, top_k=3, workspace=wl)
        return [o, l] + [r[k] for k in sorted(r)]
    alone = [once(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        both = [once(j, s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("ctx,hq,hkv", [([1500], 4, 2), ([200, 40, 0, 3000], 8, 1)])
def test_wait_budget_runs_out_cleanly(ctx, hq, hkv, monkeypatch):
    """Waits cut to one cycle give up: the kernel reports it, drains what it issued and
    returns; with a fresh workspace the next call is right."""
    from test_gpu_kv4_attention import check, problem, run
    dev = device()
    p = problem(ctx, [2] * len(ctx), hq=hq, hkv=hkv, D=128, B=16, dtype=torch.bfloat16, seed=13)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    monkeypatch.setenv("D2F_WAIT_CYCLES", "1")
    run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 5
    monkeypatch.delenv("D2F_WAIT_CYCLES")
    err.zero_()
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(p, out, lse)

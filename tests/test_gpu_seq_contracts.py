"""What the contract of d2f_prompt_attn promises about arguments that no ordinary call has."""
import ctypes

import pytest
import torch

import test_gpu_prompt_attention as prompts
import test_gpu_token_attention as tokens
from gpu_common import device
from seq_ref import check, problem

from block_causal_kv_gb300 import d2f, synth

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("cycles", [1, 100, 1000, 10000])
@pytest.mark.parametrize("D", [64, 128])
def test_waits_run_out_over_a_workspace_of_large_numbers(cycles, D, monkeypatch):
    """The composition takes no more parts than the workspace has room for, whatever the call left
    unwritten in it; the next call over it is right."""
    dev = device()
    p = problem([20, 5, 33], [4000, 300, 33], hq=2, hkv=1, D=D, B=16, dtype=BF, seed=5)
    t = prompts.to_gpu(p, dev)
    n = d2f.prompt_attn_workspace_size(3, 58, 4000, 2, 1, D, 16)
    assert n > 0
    ws = torch.full((n,), 0x7f, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    monkeypatch.setenv("D2F_WAIT_CYCLES", str(cycles))
    out, lse = prompts.call(p, t, workspace=ws, err=err)
    torch.cuda.synchronize()
    assert int(err) in (0, 5)
    if int(err) == 0:
        check(p, out, lse)
    monkeypatch.delenv("D2F_WAIT_CYCLES")
    check(p, *prompts.run(p, dev, workspace=ws))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("num_pages", [0, 4])
def test_no_pages_at_all(num_pages, dtype):
    """ctx_len of zeros over a page table without columns: there is no cache to point to."""
    dev = device()
    p = problem([150, 7], [0, 0], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=1)
    t = prompts.to_gpu(p, dev)
    want, want_lse = prompts.call(p, t)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lib = d2f.load()

    def ptr(x):
        return ctypes.c_void_p(x.data_ptr())
    status = lib.d2f_prompt_attn(ptr(t["q"]), ptr(t["k"]), ptr(t["v"]), ptr(t["start"]), None, None,
                                 None, 0, ptr(t["ctx"]), ptr(out), ptr(lse), 2, 157, 0, 4, 2, 128, 16,
                                 num_pages, d2f.BF16 if dtype == BF else d2f.F32, 1,
                                 ctypes.c_float(p["scale"]), None, 0, ptr(err),
                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert status == 0, lib.d2f_last_error_string().decode()
    assert int(err) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("batch", [2, 40, 5000])
@pytest.mark.parametrize("which", ["first", "last"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_request_without_rows_is_reported_too(dtype, which, batch):
    """A length past the page table of a request that brings no rows, in launches of one item and of
    many, while another stream keeps SMs busy."""
    dev = device()
    new = [3] * batch
    b = 0 if which == "first" else batch - 1
    new[b] = 0
    p = problem(new, [0] * batch, hq=2, hkv=2, D=64, B=16, dtype=dtype, seed=batch)
    t = prompts.to_gpu(p, dev)
    t["ctx"][b] = 10 ** 6
    busy = torch.randn((4096, 4096), device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(4):
            busy @ busy
    out, lse = prompts.call(p, t, prefix=True, max_ctx=0, err=err)
    torch.cuda.synchronize()
    assert int(err) == 1
    check(p, out, lse, rows=set(range(0, sum(new), max(1, sum(new) // 50))))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("splits", [False, True])
@pytest.mark.parametrize("what", ["negative", "decreasing", "past rows", "first", "ctx", "ctx < 0"])
def test_rows_of_skipped_requests_stay(what, splits, dtype):
    """Inconsistent lengths, with keys that are split among CTAs too: rows that only skipped requests
    own, or none, are left as they are; where row_start is consistent the other requests are right."""
    dev = device()
    p = problem([20, 30, 40], [3000 if splits else 10, 20, 33], hq=2, hkv=2, D=64, B=16, dtype=dtype,
                seed=8)
    rows = 90
    assert splits == (d2f.prompt_attn_workspace_size(3, rows, p["ctx"][0], 2, 2, 64, 16,
                                                     d2f.BF16 if dtype == BF else d2f.F32) > 0)
    t = prompts.to_gpu(p, dev)
    if what == "negative":
        t["start"][0], stay = -5, range(0, 20)
    elif what == "decreasing":                      # 0, 20, 10, 10
        t["start"][2:], stay = 10, range(20, 90)
    elif what == "past rows":
        t["start"][3], stay = 91, range(50, 90)
    elif what == "first":
        t["start"][0], stay = 5, range(0, 5)
    else:
        t["ctx"][1] = p["table"].shape[1] * 16 + 1 if what == "ctx" else -1
        stay = range(20, 50)
    out = torch.full((rows, 2, 64), 7.0, dtype=dtype, device=dev)
    lse = torch.full((rows, 2), 7.0, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    prompts.call(p, t, err=err, out=out, lse=lse, max_ctx=p["ctx"][0])
    torch.cuda.synchronize()
    assert int(err) == 1
    stay = torch.tensor(list(stay), device=dev)
    assert bool((out[stay] == 7).all()) and bool((lse[stay] == 7).all())
    if what.startswith("ctx"):
        p["ctx"][1] = -1
        check(p, out, lse)


def test_a_workspace_zeroed_between_entry_points_that_do_not_share_one():
    """Calls whose counters pass four an SM (a commit of many blocks, a window attention with num_splits
    given) use a prompt's or a single token's workspace once it is zeroed again, and it theirs."""
    dev = device()
    w = synth.Workload("m", 4, 1, 1, 8, 1, BF, [0] * 4, [640, 400, 960, 240], 96, masked_frac=0.6,
                       taus=(0.05, 0.3, 0.6), logit_sigma=1.5, seed=3)
    c = synth.make_problem(w)

    def commit(ws):
        g = c.to(dev)
        res = d2f.commit(g.logits, g.tokens, g.masked, g.q_start, g.block_phase, g.tau, block_size=1,
                         mask_id=c.mask_id, num_splits=2, workspace=ws)
        return g.tokens, g.masked, res["conf"], res["argmax"], res["block_remaining"]
    w = synth.Workload("w", 24, 32, 32, 128, 16, F32, [64] * 24, [1] * 24, 64, permute_pages=True,
                       seed=4)
    a = synth.make_problem(w)
    g = a.to(dev)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    assert 24 * 32 > 4 * sms and 2 * 2240 > 4 * sms

    def windows(ws):
        return d2f.block_attn(g.q, g.k_win, g.v_win, g.k_pool, g.v_pool, g.page_table, g.ctx_len,
                              g.q_start, block_size=16, max_q_per_seq=a.max_q_per_seq,
                              max_ctx=a.max_ctx, num_splits=2, workspace=ws)
    p = problem([200, 9], [2200, 100], hq=2, hkv=1, D=128, B=16, dtype=F32, seed=1)
    t = prompts.to_gpu(p, dev)
    q = tokens.batch([3000, 5, 700], hq=8, hkv=2, D=128, B=16, dtype=BF, seed=2)
    u = tokens.to_gpu(q, dev)
    calls = [(commit, d2f.commit_workspace_size(2240, 96, 1, num_splits=2)),
             (windows, d2f.attn_workspace_size(24, w.total_q, a.max_q_per_seq, a.max_ctx, 32, 32, 128,
                                               16, d2f.F32, 2)),
             (lambda ws: prompts.call(p, t, workspace=ws),
              d2f.prompt_attn_workspace_size(2, 209, 2200, 2, 1, 128, 16, d2f.F32)),
             (lambda ws: tokens.call(q, u, workspace=ws),
              d2f.token_attn_workspace_size(3, 3000, 8, 2, 128, 16))]
    assert all(n > 4 * 4 * sms for _, n in calls)
    fresh = [[x.clone() for x in f(torch.zeros(n, dtype=torch.uint8, device=dev))] for f, n in calls]
    ws = torch.zeros(max(n for _, n in calls), dtype=torch.uint8, device=dev)
    for i in (2, 0, 3, 1, 2, 3, 0, 1, 3, 0, 2, 1):
        ws.zero_()
        for got, want in zip(calls[i][0](ws), fresh[i]):
            assert torch.equal(got, want), i


@pytest.mark.parametrize("hq", [65, 127, 128, 129])
@pytest.mark.parametrize("D,B", [(128, 8), (64, 128)])
@pytest.mark.parametrize("new,ctx", [([5, 1, 40], [0, 0, 0]), ([3, 0, 9], [1500, 7, 130])])
def test_groups_about_a_row_tile_wide(new, ctx, D, B, hq):
    """One query, or none beside another, in a tile of 128 rows; one head more than a tile has."""
    dev = device()
    p = problem(new, ctx, hq=hq, hkv=1, D=D, B=B, dtype=BF, seed=hq)
    check(p, *prompts.run(p, dev))
    p = tokens.batch([c + 1 for c in ctx], hq=hq, hkv=1, D=D, B=B, dtype=BF, seed=hq)
    check(p, *tokens.run(p, dev))

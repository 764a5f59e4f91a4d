"""d2f_prompt_attn, d2f_token_attn and d2f_kv_store at their edges: waits that run out, scores at the
ends of float, offsets past 32 bits, large batches, shared pages, shared workspaces, other streams,
several threads, and writes outside their buffers."""
import numpy as np
import pytest
import torch

import test_gpu_prompt_attention as prompts
import test_gpu_streams as streams
import test_gpu_token_attention as tokens
from gpu_common import device
from seq_ref import check, problem
from test_gpu_errors import _canary_intact, _guarded, _guarded_like
from test_gpu_threads import together
from test_gpu_workspaces import attention_call, check_sequence, logprobs_call, workspace

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TIMEOUT = 5


def dt(dtype):
    return d2f.BF16 if dtype == BF else d2f.F32


def prompt_size(p):
    rows, hq, D = p["q"].shape
    return d2f.prompt_attn_workspace_size(len(p["ctx"]), rows, max(p["ctx"]), hq, p["k"].shape[1], D,
                                          p["B"], dt(p["dtype"]))


def token_size(p):
    n, hq, D = p["q"].shape
    return d2f.token_attn_workspace_size(n, max(p["ctx"]), hq, p["k"].shape[1], D, p["B"],
                                         dt(p["dtype"]))


@pytest.mark.parametrize("cycles", [1, 300, 3000, 30000])
@pytest.mark.parametrize("splits", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_waits_of_prompts_run_out(cycles, splits, D, monkeypatch):
    """Waits that give up sooner or later in the call: it returns and reports them if there were any,
    and the next call is right."""
    dev = device()
    p = problem([300, 5, 130], [0, 1500 if splits else 300, 33], hq=2, hkv=1, D=D, B=16, dtype=BF,
                seed=5)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    t = prompts.to_gpu(p, dev)
    torch.cuda.synchronize()
    monkeypatch.setenv("D2F_WAIT_CYCLES", str(cycles))
    out, lse = prompts.call(p, t, err=err)
    torch.cuda.synchronize()
    assert int(err) in (0, TIMEOUT) and (cycles > 1 or int(err) == TIMEOUT)
    if int(err) == 0:
        check(p, out, lse)
    monkeypatch.delenv("D2F_WAIT_CYCLES")
    check(p, *prompts.run(p, dev))


@pytest.mark.parametrize("path", ["", "simt"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ctx", [3, 40, 2500])
def test_scores_at_the_ends_of_float(ctx, dtype, path, monkeypatch):
    """Very low scores with the largest at one key, whose V is the output; scores of -infinity, which
    have no weight; rows with no other score, whose output is 0."""
    if path:
        monkeypatch.setenv("D2F_ATTN_PATH", path)
    dev = device()
    for n, mod, run in ((150, prompts, prompts.run), (1, tokens, tokens.run)):
        tc = dtype == BF and not path
        # the scores go down to -5e8, as far as prompts on the tensor cores take them, or -2.5e33
        low = 4e9 if tc and mod is prompts else 2e34
        p = problem([n], [ctx], hq=2, hkv=1, D=64, B=16, dtype=dtype, seed=ctx)
        p["mask_block"] = 0
        best = ctx // 2
        for x in ("q", "k", "k_pool"):
            p[x].zero_()
        p["q"][..., 0] = 1.0
        p["k"][..., 0] = -low / 2
        p["k_pool"][..., 0] = -low
        p["k_pool"][p["table"][0, best // 16], 0, best % 16, 0] = -low / 4
        out, lse = run(p, dev)
        want = p["v_pool"][p["table"][0, best // 16], 0, best % 16].double()
        top = p["scale"] * float(p["k_pool"][p["table"][0, best // 16], 0, best % 16, 0].double())
        # one weight, rounded to bf16 on the tensor cores, and the output's rounding
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * 2 if tc else 2.0 ** -22
        assert bool(((out.cpu().double() - want).abs() <= tol * want.abs()).all())
        # (float32 products and logarithms: a few roundings of 2^-24)
        assert np.allclose(lse.cpu().double().numpy(), top, rtol=1e-6, atol=0)
        # -infinity: none of the new keys, then none at all
        p["k_pool"][..., 0] = 0.5
        p["k"][..., 0] = float("-inf")
        out, lse = run(p, dev)
        check(p, out, lse, see_new=False)
        p["k_pool"][..., 0] = float("-inf")
        out, lse = run(p, dev)
        assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("hq,hkv,D,B", [(4, 2, 128, 16), (3, 1, 64, 8), (16, 1, 128, 32)])
def test_bf16_on_the_cuda_cores(hq, hkv, D, B, monkeypatch):
    monkeypatch.setenv("D2F_ATTN_PATH", "simt")
    dev = device()
    p = problem([70, 1, 0, 129], [0, 1300, 7, 64], hq=hq, hkv=hkv, D=D, B=B, dtype=BF, seed=1)
    check(p, *prompts.run(p, dev))
    p = tokens.batch([0, 1, 2100, 64, 63], hq=hq, hkv=hkv, D=D, B=B, dtype=BF, seed=2)
    check(p, *tokens.run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,hkv", [(1024, 4), (1025, 4), (700, 8), (1023, 1)])
def test_batches_of_about_a_thousand(n, hkv, dtype):
    """Where the tensor-core path takes whole (sequence, KV head)s instead of runs of its line."""
    dev = device()
    g = torch.Generator().manual_seed(n)
    ctx = torch.randint(-20, 90, (n,), generator=g).tolist()
    ctx[5] = 3000
    p = tokens.batch(ctx, hq=hkv, hkv=hkv, D=64, B=16, dtype=dtype, seed=n)
    out, lse = torch.zeros_like(p["q"]).to(dev), torch.zeros(p["q"].shape[:2], device=dev)
    check(p, *tokens.run(p, dev, out=out, lse=lse))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_that_sequences_share(dtype):
    """The same first pages in every table row, once the same page twice in a row."""
    dev = device()
    p = problem([40, 3, 70], [96, 100, 130], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=3)
    p["table"][1, :6] = p["table"][0, :6]
    p["table"][2, :4] = p["table"][0, [0, 1, 1, 0]]
    check(p, *prompts.run(p, dev))
    p = tokens.batch([100, 97, 130], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=3)
    p["table"][1, :6] = p["table"][0, :6]
    p["table"][2, :4] = p["table"][0, [0, 1, 1, 0]]
    check(p, *tokens.run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pools_past_32_bits(dtype):
    """Pages whose elements lie past 2^32 of a pool."""
    dev = device()
    B, D = 16, 128
    pages = (1 << 32) // (2 * B * D) + 9
    big = torch.empty((pages, 2, B, D), dtype=dtype, device=dev)
    for n, mod in ((20, prompts), (1, tokens)):
        p = problem([n, n], [90, 1200], hq=4, hkv=2, D=D, B=B, dtype=dtype, seed=7)
        p["mask_block"] = 0
        p["v_pool"] = p["k_pool"].clone()   # one pool for both
        used = p["k_pool"].shape[0]
        g = torch.Generator().manual_seed(1)
        at = torch.cat([torch.arange(pages - 8, pages), torch.randint(0, pages - 8, (used - 8,),
                                                                      generator=g).unique()])
        at = torch.cat([at, torch.arange(used - len(at))]) if len(at) < used else at
        assert len(at.unique()) == used
        big[at.to(dev)] = p["k_pool"].to(dev)
        t = mod.to_gpu(p, dev)
        t["table"] = torch.from_numpy(np.where(p["table"] < 0, -1, at.numpy()[p["table"]])
                                      .astype(np.int32)).to(dev)
        t["k_pool"] = t["v_pool"] = big
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        kw = {} if mod is prompts else dict(new=False)
        out, lse = mod.call(p, t, err=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        check(p, out, lse, see_new=mod is prompts)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_past_32_bits(dtype):
    """Queries and outputs whose elements lie past 2^32."""
    dev = device()
    hq, D, n = 64, 128, 9
    batch = (1 << 32) // (hq * D * n) + 3
    rows = batch * n
    g = torch.Generator(device=dev).manual_seed(2)
    q = torch.empty((rows, hq, D), dtype=dtype, device=dev).normal_(generator=g)
    k, v = (torch.randn((rows, 1, D), generator=g, device=dev).to(dtype) for _ in range(2))
    start = torch.arange(0, rows + 1, n, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = d2f.prompt_attn(q, k, v, start, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for b in (0, batch // 2, batch - 2, batch - 1):
        r = slice(b * n, (b + 1) * n)
        p = problem([n], [0], hq=hq, hkv=1, D=D, B=16, dtype=dtype, seed=1)
        p.update(q=q[r].cpu(), k=k[r].cpu(), v=v[r].cpu())
        check(p, out[r], lse[r])
    del out, lse, q
    # single tokens: as many sequences as there may be, 513 heads
    batch, hq = 65535, 513
    q = torch.empty((batch, hq, D), dtype=dtype, device=dev).normal_(generator=g)
    assert q.numel() > 1 << 32
    pool = torch.randn((4, 1, 16, D), generator=g, device=dev).to(dtype)
    table = torch.zeros((batch, 1), dtype=torch.int32, device=dev)
    ctx = torch.full((batch,), 5, dtype=torch.int32, device=dev)
    table[-2:, 0] = torch.tensor([3, 1], dtype=torch.int32)
    out, lse = d2f.token_attn(q, pool, pool, table, ctx, block_size=16, max_ctx=5, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for b, page in ((0, 0), (batch // 2, 0), (batch - 2, 3), (batch - 1, 1)):
        p = problem([1], [5], hq=hq, hkv=1, D=D, B=16, dtype=dtype, seed=1)
        p.update(q=q[b:b + 1].cpu(), k_pool=pool.cpu(), v_pool=pool.cpu(),
                 table=np.array([[page]], np.int32))
        check(p, out[b:b + 1], lse[b:b + 1], see_new=False)


def prompt_call(p, dev):
    t = prompts.to_gpu(p, dev)
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device=dev)

    def call(ws):
        out.fill_(7)
        lse.fill_(7)
        prompts.call(p, t, out=out, lse=lse, workspace=ws)
        return out, lse
    return call, prompt_size(p)


def token_call(p, dev):
    t = tokens.to_gpu(p, dev)
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device=dev)

    def call(ws):
        out.fill_(7)
        lse.fill_(7)
        tokens.call(p, t, out=out, lse=lse, workspace=ws)
        return out, lse
    return call, token_size(p)


def calls(dtype, dev):
    from test_gpu_kv4_attention import problem as kv4_problem
    kw = dict(D=128, B=16, dtype=dtype)
    return [
        prompt_call(problem([20, 9], [2200, 100], hq=2, hkv=1, seed=1, **kw), dev),
        token_call(tokens.batch([3000, 5, 700], hq=8, hkv=2, seed=2, **kw), dev),
        token_call(tokens.batch([900] * 9, hq=32, hkv=32, seed=3, **kw), dev),
        token_call(tokens.batch([130] * 20, hq=40, hkv=40, seed=4, **kw), dev),
        attention_call(kv4_problem([2100], [1], hq=4, hkv=4, seed=1, **kw), dev),
        logprobs_call(3, 60000, dtype, 5, dev),
        prompt_call(problem([1], [3000], hq=4, hkv=4, seed=5, **kw), dev),
    ]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_workspace_for_all(dtype):
    dev = device()
    check_sequence(calls(dtype, dev), [0, 1, 4, 2, 6, 5, 3, 1, 0, 3, 2, 5, 4, 0, 1], dev)


def test_several_threads():
    dev = device()
    todo = calls(BF, dev) + calls(F32, dev)
    torch.cuda.synchronize()

    def job(call, size):
        def body():
            with torch.cuda.stream(torch.cuda.Stream()):
                ws = workspace(max(size, 1), dev)
                first = [x.clone() for x in call(ws)]
                for _ in range(200):
                    got = call(ws)
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(first, got))
        return body
    together([job(*c) for c in todo])


NAMES = ["prompt bf16", "prompt f32", "token bf16", "token f32"]


def make(name, dev):
    """(call(stream) -> the tensors it made, bytes of its workspace)."""
    kw = dict(hq=8, hkv=8, D=128, B=16, dtype=BF if name.endswith("bf16") else F32, seed=1)
    if name.startswith("prompt"):
        p = problem([16], [2100], **kw)
        t = prompts.to_gpu(p, dev)
        return lambda s: prompts.call(p, t, stream=s), prompt_size(p)
    p = tokens.batch([2100, 700], **kw)
    t = tokens.to_gpu(p, dev)
    return lambda s: tokens.call(p, t, stream=s), token_size(p)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("what", ["workspace_made_behind_a_busy_current_stream",
                                  "results_share_no_memory_with_pending_work",
                                  "results_stay_the_callers_until_it_is_done",
                                  "captured_on_a_forked_stream"])
def test_streams(what, name, monkeypatch):
    """What test_gpu_streams.py asks of the other entry points."""
    monkeypatch.setattr(streams, "make", make)
    args = (name, monkeypatch) if "busy" in what else (name,)
    getattr(streams, "test_" + what)(*args)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D,B", [(4, 2, 128, 16), (5, 1, 64, 8), (2, 2, 32, 16), (71, 1, 128, 16)])
@pytest.mark.parametrize("ctx", [70, 2300])
def test_writes_stay_inside_their_buffers(ctx, hq, hkv, D, B, dtype):
    dev = device()
    p = problem([33, 1, 150], [ctx, 0, 17], hq=hq, hkv=hkv, D=D, B=B, dtype=dtype, seed=1)
    q = tokens.batch([ctx, 0, 17, ctx + 1], hq=hq, hkv=hkv, D=D, B=B, dtype=dtype, seed=2)
    for p, mod, size in ((p, prompts, prompt_size(p)), (q, tokens, token_size(q))):
        t = mod.to_gpu(p, dev)
        pools = {x: _guarded_like(p[x].shape, dtype, dev) for x in ("k_pool", "v_pool")}
        for x in pools:
            pools[x][1].copy_(t[x])
            t[x] = pools[x][1]
        o, out = _guarded_like(t["q"].shape, dtype, dev, 7)
        l, lse = _guarded_like(t["q"].shape[:2], F32, dev, 7)
        w, ws = _guarded(max(size, 16), dev)
        ws.zero_()
        mod.call(p, t, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        for buf, label in ((o, "out"), (l, "lse"), (w, "workspace"), (pools["k_pool"][0], "K"),
                           (pools["v_pool"][0], "V")):
            _canary_intact(buf, label)
        check(p, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompts_of_one_row(dtype):
    """A batch of prompts of one row each is what single tokens compute."""
    dev = device()
    p = tokens.batch([0, 1, 15, 16, 400, 2000], hq=8, hkv=2, D=128, B=16, dtype=dtype, seed=8)
    check(p, *prompts.run(dict(p, mask_block=1), dev))
    check(p, *tokens.run(p, dev))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,ctx", [
    ([1, 30, 5, 66, 2, 0, 9], [9000, 0, 8192, 300, 127, 4000, 2500]),
    ([2] * 9 + [40], [8200] * 10),                       # as long as one another: nothing is split
    ([1] * 95 + [3], [0, 17] * 47 + [9000, 260]),        # the largest batch that is split
    ([1] * 96 + [3], [0, 17] * 48 + [9000]),             # one more
    ([1, 1], [20000, 0]),
    ([130, 1, 70], [8300, 8300, 8400])])
def test_keys_of_uneven_requests(new, ctx, D):
    """Splits that the device chooses: requests with many, with one, and with none."""
    dev = device()
    p = problem(new, ctx, hq=4, hkv=2, D=D, B=16, dtype=BF, seed=len(new), mask_block=16)
    rows = {int(r) for r in np.random.default_rng(1).choice(sum(new), min(sum(new), 60), False)}
    out, lse = prompts.run(p, dev)
    check(p, out, lse, rows)
    again = prompts.run(p, dev, max_ctx=0)   # (the hint shapes the splits, nothing else)
    check(p, *again, rows)


@pytest.mark.parametrize("mask_block", [1, 0, 1000])
@pytest.mark.parametrize("D,B", [(64, 128), (128, 128), (128, 8)])
def test_prompts_whose_tiles_end_apart(D, B, mask_block):
    """The two row tiles of an item see numbers of keys that lie far apart, pages as long as a tile, more
    items than CTAs, whole tiles of bad pages between good ones: the same bits every time."""
    dev = device()
    g = np.random.default_rng(D + B + mask_block)
    new = [1100, 90, 1, 700, 2300, 40] * 4
    ctx = [0, 700, 1500, 130, 5, 1030] * 4
    p = problem(new, ctx, hq=12, hkv=6, D=D, B=B, dtype=BF, seed=3, mask_block=mask_block)
    pages = p["k_pool"].shape[0]
    p["table"][2, 256 // B:768 // B] = pages + 5
    p["table"][5, :256 // B] = -4
    rows = {int(r) for r in g.choice(sum(new), 40, False)}
    rows |= {int(p["start"][b]) for b in (2, 5)}
    t = prompts.to_gpu(p, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = prompts.call(p, t, err=err)
    torch.cuda.synchronize()
    assert int(err) == 4   # the bad pages
    check(p, out, lse, rows)
    for _ in range(30):
        err.zero_()
        again = prompts.call(p, t, err=err)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and int(err) == 4

"""d2f_prompt_attn against float64 attention, with elementwise error bounds (tests/seq_ref.py)."""
import numpy as np
import pytest
import torch

from gpu_common import device
from seq_ref import check, problem

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def to_gpu(p, dev):
    t = {k: p[k].to(dev) for k in ("q", "k", "v", "k_pool", "v_pool")}
    t["table"] = torch.from_numpy(p["table"]).to(dev)
    t["ctx"] = torch.tensor(p["ctx"], dtype=torch.int32, device=dev)
    t["start"] = torch.from_numpy(p["start"]).to(dev)
    return t


def call(p, t, *, prefix=None, max_ctx=None, **kw):
    if prefix is None:
        prefix = any(p["ctx"])
    more = {} if not prefix else dict(
        k_pool=t["k_pool"], v_pool=t["v_pool"], page_table=t["table"], ctx_len=t["ctx"],
        max_ctx=max(p["ctx"]) if max_ctx is None else max_ctx)
    return d2f.prompt_attn(t["q"], t["k"], t["v"], t["start"], mask_block=p["mask_block"],
                           block_size=p["B"], softmax_scale=p["scale"], **more, **kw)


def run(p, dev, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = call(p, to_gpu(p, dev), err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, lse


SHAPES = [  # hq, hkv, D, B
    (4, 4, 128, 16), (4, 4, 64, 16), (8, 2, 128, 8), (14, 2, 128, 16), (5, 1, 64, 32),
    (2, 2, 32, 16), (3, 1, 128, 5), (4, 2, 64, 1), (2, 1, 32, 256), (71, 1, 64, 16),
    (130, 1, 128, 32), (6, 2, 128, 128),
]
LENS = [1, 0, 2, 31, 64, 65, 127, 128, 129, 0, 260, 300]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D,B", SHAPES)
def test_packed_causal(hq, hkv, D, B, dtype):
    """Requests of none, one row, a tile less one, whole tiles, odd ends."""
    dev = device()
    lens = LENS if hq < 70 else [1, 0, 3, 129]
    p = problem(lens, [0] * len(lens), hq=hq, hkv=hkv, D=D, B=B, dtype=dtype, seed=hq + D + B)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask_block", [0, 1, 2, 7, 16, 32, 100, 128, 1000])
def test_mask_blocks(mask_block, dtype):
    dev = device()
    p = problem([1, 15, 16, 17, 130, 301], [0, 40, 16, 0, 129, 3], hq=4, hkv=2, D=128, B=16,
                dtype=dtype, seed=mask_block, mask_block=mask_block)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D,B", SHAPES)
def test_behind_a_prefix(hq, hkv, D, B, dtype):
    """Cached prefixes of no token, one, a page less one, whole pages and tiles, odd ends."""
    dev = device()
    ctx = [0, 1, B - 1, B, 127, 128, 129, 300, 700]
    new = [3, 1, 2, 40, 0, 17, 1, 129, 5]
    if hq >= 70:
        ctx, new = ctx[4:], [1, 2, 0, 1, 3]
    p = problem(new, ctx, hq=hq, hkv=hkv, D=D, B=B, dtype=dtype, seed=hq * 3 + D + B, mask_block=4)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D,n,ctx", [
    (4, 1, 128, [1], [5000]), (7, 1, 128, [40, 3], [3000, 4097]), (2, 2, 64, [1, 1, 1], [0, 2500, 9]),
    (28, 4, 128, [17], [1500]), (2, 2, 32, [70], [1100])])
def test_few_rows_behind_long_prefixes(hq, hkv, D, n, ctx, dtype):
    """The keys are split among CTAs."""
    dev = device()
    p = problem(n, ctx, hq=hq, hkv=hkv, D=D, B=16, dtype=dtype, seed=sum(ctx))
    w = d2f.prompt_attn_workspace_size(len(n), sum(n), max(ctx), hq, hkv, D, 16,
                                       d2f.BF16 if dtype == BF else d2f.F32)
    assert w > 0  # split
    check(p, *run(p, dev))
    # the hint only shapes the split
    check(p, *run(p, dev, max_ctx=0))


@pytest.mark.parametrize("dtype,hq,hkv,D,n,mask_block", [
    (BF, 2, 2, 128, 2100, 1), (BF, 7, 1, 128, 1500, 1), (BF, 4, 1, 64, 3000, 32),
    (BF, 1, 1, 128, 2500, 0), (F32, 2, 1, 64, 1500, 1), (BF, 2, 2, 128, 9000, 1)])
def test_long_prompts(dtype, hq, hkv, D, n, mask_block):
    dev = device()
    p = problem([n, 5], [0, 0], hq=hq, hkv=hkv, D=D, B=16, dtype=dtype, seed=n, q_scale=2.0,
                mask_block=mask_block)
    some = set(range(0, n, 97)) | {1, 127, 128, 255, 256, 257, n - 1, n, n + 4}
    check(p, *run(p, dev), rows=some)


def test_many_requests():
    """More requests than one step of the tile search probes, most of them short."""
    dev = device()
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 9, (1500,), generator=g).tolist()
    lens[700], lens[1499] = 400, 0
    p = problem(lens, [0] * 1500, hq=2, hkv=1, D=64, B=16, dtype=BF, seed=5, spare=0)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_flat_and_sharp_softmax(scale, dtype):
    """Nearly equal weights; one weight that takes nearly all, maxima that keep growing."""
    dev = device()
    p = problem([200, 140], [0, 260], hq=2, hkv=2, D=128, B=16, dtype=dtype, seed=9, q_scale=scale)
    if scale > 1:   # keys that grow along the prompt: every tile moves the reference
        ramp = torch.linspace(0.2, 1.0, p["k"].shape[0])[:, None, None]
        p["k"] = (p["k"].float() * ramp).to(dtype)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_hidden_keys_do_not_reach_a_row(value, dtype):
    """Infinite and NaN K and V of later rows, of another request, behind the last request and in
    slots past the context reach the rows that see them only."""
    dev = device()
    new, ctx = [150, 3, 290, 20], [0, 37, 130, 0]
    p = problem(new, ctx, hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=4, tail=30)
    s = p["start"]
    p["v"][s[0] + 100, 0, 5] = value           # inside the first request's diagonal tile
    p["v"][s[1]:s[2]] = value                  # all of the second
    p["k"][s[2] + 200, 1, 3] = value           # a later key of the third
    p["v"][s[2] + 210, 1] = value
    p["k"][s[4]:], p["v"][s[4]:], p["q"][s[4]:] = value, value, value
    for b, c in enumerate(ctx):                # slots past the context
        if c % 16:
            p["k_pool"][p["table"][b, c // 16], :, c % 16:] = value
            p["v_pool"][p["table"][b, c // 16], :, c % 16:] = value
    unused = set(range(p["k_pool"].shape[0])) - set(p["table"].flatten().tolist())
    for page in unused:
        p["k_pool"][page] = value
        p["v_pool"][page] = value
    check(p, *run(p, dev))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_odd_cached_values_reach_every_row(value):
    dev = device()
    p = problem([9, 140], [40, 300], hq=2, hkv=2, D=64, B=16, dtype=BF, seed=4)
    p["v_pool"][p["table"][0, 1], 0, 3, 7] = value
    p["v_pool"][p["table"][1, 9], 1, 0, :9] = value
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype,splits", [(BF, False), (F32, False), (BF, True), (F32, True)])
def test_rows_behind_the_last_request_stay(dtype, splits):
    dev = device()
    p = problem([20, 7], [2000, 33] if splits else [0, 33], hq=2, hkv=1, D=128, B=16, dtype=dtype,
                seed=8, tail=50)
    out = torch.full_like(p["q"], 7.0).to(dev)
    lse = torch.full(p["q"].shape[:2], 7.0, device=dev)
    check(p, *run(p, dev, out=out, lse=lse))
    n = int(p["start"][-1])
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_pages_are_left_out(dtype):
    dev = device()
    p = problem([30, 150, 4], [70, 200, 16], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=2)
    p["v_pool"][0] = float("nan")              # (a wild id must not end up here)
    p["table"][p["table"] == 0] = p["k_pool"].shape[0] - 1
    p["table"][0, 2] = -3
    p["table"][1, 0] = p["k_pool"].shape[0]
    p["table"][1, 12] = 2 ** 31 - 1
    p["table"][2, 0] = -1                      # the whole prefix
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = call(p, to_gpu(p, dev), err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["negative", "decreasing", "past rows", "first", "ctx", "ctx < 0"])
def test_inconsistent_lengths(what, dtype):
    """Reported; requests with such lengths are skipped, nothing outside the buffers is written."""
    dev = device()
    p = problem([20, 30, 40], [10, 20, 33], hq=2, hkv=2, D=64, B=16, dtype=dtype, seed=8)
    t = to_gpu(p, dev)
    skipped = [1]
    if what == "negative":
        t["start"][0], skipped = -5, [0]
    elif what == "decreasing":
        t["start"][2], skipped = 10, [1, 2]
    elif what == "past rows":
        t["start"][3], skipped = 91, [2]
    elif what == "first":
        t["start"][0], skipped = 5, [0]
    elif what == "ctx":
        t["ctx"][1] = p["table"].shape[1] * 16 + 1
    else:
        t["ctx"][1] = -1
    pad = 64
    whole = torch.full((90 + 2 * pad, 2, 64), 7.0, dtype=dtype, device=dev)
    lses = torch.full((90 + 2 * pad, 2), 7.0, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    call(p, t, err=err, out=whole[pad:-pad], lse=lses[pad:-pad], max_ctx=33)
    torch.cuda.synchronize()
    assert int(err) == 1
    for x in (whole, lses):
        assert bool((x[:pad] == 7).all()) and bool((x[-pad:] == 7).all())
    if what in ("ctx", "ctx < 0"):
        assert bool((whole[pad + 20:pad + 50] == 7).all())
        p["ctx"][1] = -1
        check(p, whole[pad:-pad], lses[pad:-pad])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("splits", [False, True])
def test_repeats_capture_and_streams(dtype, splits):
    """The same bits from every call: again, on another stream, captured and replayed with lengths
    that changed on the device, with a workspace that other calls used."""
    dev = device()
    p = problem([60, 3, 140], [0, 2200 if splits else 50, 33], hq=2, hkv=1, D=128, B=16, dtype=dtype,
                seed=6)
    t = to_gpu(p, dev)
    n = d2f.prompt_attn_workspace_size(3, 203, max(p["ctx"]), 2, 1, 128, 16,
                                       d2f.BF16 if dtype == BF else d2f.F32)
    assert (n > 0) == splits
    ws = torch.randint(0, 255, (max(n, 1),), dtype=torch.uint8, device=dev)  # (needs no zeroing)
    first = [x.clone() for x in call(p, t, workspace=ws)]
    check(p, *first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for again in (call(p, t, workspace=ws), call(p, t), call(p, t, stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, t, workspace=ws, out=out, lse=lse)
    for new, ctx in (([60, 3, 140], p["ctx"]), ([3, 150, 50], [7, 0, p["ctx"][1]])):
        if ctx[2] > p["table"].shape[1] * 16:
            continue
        q = dict(p, new=new, ctx=ctx, start=np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        need = [-(-c // 16) for c in ctx]
        if max(need) > p["table"].shape[1] or sum(need) > p["k_pool"].shape[0]:
            continue
        table, at = np.full_like(p["table"], -1), 0
        for b, m in enumerate(need):
            table[b, :m] = np.arange(at, at + m)
            at += m
        if new != p["new"]:
            q["table"] = table
        t["start"].copy_(torch.from_numpy(q["start"]))
        t["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        t["table"].copy_(torch.from_numpy(q["table"]))
        graph.replay()
        torch.cuda.synchronize()
        check(q, out, lse)


def test_nothing_to_do():
    dev = device()
    p = problem([0, 0], [5, 0], hq=2, hkv=1, D=64, B=16, dtype=BF, seed=1)
    out, lse = run(p, dev)
    assert out.shape[0] == 0 and lse.shape[0] == 0


def test_refusals():
    dev = device()
    p = problem([20], [30], hq=4, hkv=2, D=64, B=16, dtype=BF, seed=1)
    t = to_gpu(p, dev)
    for key, bad in (("q", t["q"].float()), ("k", t["k"][:, :1]), ("v", t["v"].transpose(0, 1)),
                     ("k", t["k"].cpu()), ("k_pool", t["k_pool"][:, :, :8]),
                     ("table", t["table"].long()), ("ctx", t["ctx"][:0]),
                     ("start", t["start"].float())):
        with pytest.raises((ValueError, TypeError, d2f.D2FError)):
            call(p, dict(t, **{key: bad}))
    for kw in (dict(max_ctx=10 ** 6), dict(out=t["q"][:-1])):
        with pytest.raises((ValueError, d2f.D2FError)):
            call(p, t, **kw)
    table = torch.zeros((1, 500), dtype=torch.int32, device=dev)
    for ws in (torch.zeros(64, dtype=torch.uint8, device=dev),                    # too small
               torch.zeros(1 << 24, dtype=torch.uint8, device=dev)[8:]):          # not aligned
        with pytest.raises(d2f.D2FError):
            call(p, dict(t, table=table), max_ctx=8000, workspace=ws)
    with pytest.raises(ValueError):
        d2f.prompt_attn(t["q"], t["k"], t["v"], t["start"], ctx_len=t["ctx"])
    with pytest.raises(d2f.D2FError):   # a prefix hint without a prefix
        d2f.prompt_attn(t["q"], t["k"], t["v"], t["start"], max_ctx=16)

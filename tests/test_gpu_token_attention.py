"""d2f_token_attn against float64 attention, with elementwise error bounds (tests/seq_ref.py)."""
import numpy as np
import pytest
import torch

from gpu_common import device
from seq_ref import check, problem

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def batch(ctx, **kw):
    p = problem([1] * len(ctx), ctx, **kw)
    p["mask_block"] = 0
    return p


def to_gpu(p, dev):
    t = {k: p[k].to(dev) for k in ("q", "k", "v", "k_pool", "v_pool")}
    t["table"] = torch.from_numpy(p["table"]).to(dev)
    t["ctx"] = torch.tensor(p["ctx"], dtype=torch.int32, device=dev)
    return t


def call(p, t, *, new=True, max_ctx=None, **kw):
    more = dict(k_new=t["k"], v_new=t["v"]) if new else {}
    return d2f.token_attn(t["q"], t["k_pool"], t["v_pool"], t["table"], t["ctx"],
                          block_size=p["B"], max_ctx=max(max(p["ctx"]), 0) if max_ctx is None else max_ctx,
                          softmax_scale=p["scale"], **more, **kw)


def pools_after(p):
    """The pools with every sequence's new token in its slot."""
    kp, vp = p["k_pool"].clone(), p["v_pool"].clone()
    for b, c in enumerate(p["ctx"]):
        if c < 0 or c // p["B"] >= p["table"].shape[1]:
            continue
        page = int(p["table"][b, c // p["B"]])
        if 0 <= page < kp.shape[0]:
            kp[page, :, c % p["B"]], vp[page, :, c % p["B"]] = p["k"][b], p["v"][b]
    return kp, vp


def bits(x):
    return x.cpu().contiguous().view(torch.uint8)


def run(p, dev, **kw):
    t = to_gpu(p, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    new = kw.get("new", True)
    out, lse = call(p, t, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    kp, vp = pools_after(p) if new else (p["k_pool"], p["v_pool"])
    assert torch.equal(bits(t["k_pool"]), bits(kp)) and torch.equal(bits(t["v_pool"]), bits(vp))
    return out, lse


SHAPES = [  # hq, hkv, D, B
    (4, 4, 128, 16), (4, 4, 64, 16), (8, 2, 128, 8), (14, 2, 128, 16), (5, 1, 64, 32),
    (2, 2, 32, 16), (3, 1, 128, 5), (4, 2, 64, 1), (2, 1, 32, 256), (71, 1, 64, 16),
    (17, 1, 128, 16), (16, 1, 128, 128), (6, 2, 128, 256), (2, 2, 128, 1),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("hq,hkv,D,B", SHAPES)
def test_ragged_batch(hq, hkv, D, B, new, dtype):
    """Contexts of no token, one, a page less one, whole pages and tiles, odd ends; sequences that
    take no part."""
    dev = device()
    p = batch([0, 1, B - 1, B, B + 1, -1, 63, 64, 65, 127, 128, 700, -7, 0], hq=hq, hkv=hkv, D=D, B=B,
              dtype=dtype, seed=hq + D + B)
    out = torch.full_like(p["q"], 7.0).to(dev)
    lse = torch.full(p["q"].shape[:2], 7.0, device=dev)
    check(p, *run(p, dev, new=new, out=out, lse=lse), see_new=new)
    for b in (5, 12):
        assert bool((out[b] == 7).all()) and bool((lse[b] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D,ctx", [
    (4, 1, 128, [9000]), (7, 1, 128, [3000, 4097, 0]), (2, 2, 64, [0, 12500, 9]),
    (28, 4, 128, [1500]), (2, 2, 32, [5100]), (4, 4, 128, [1] * 40 + [6000] + [2] * 30),
    (40, 2, 128, [2600, 700])])
def test_long_contexts(hq, hkv, D, ctx, dtype):
    """The cache's length is split among CTAs; the hint only shapes the split."""
    dev = device()
    p = batch(ctx, hq=hq, hkv=hkv, D=D, B=16, dtype=dtype, seed=sum(ctx), q_scale=1.5)
    check(p, *run(p, dev))
    check(p, *run(p, dev, max_ctx=0))
    check(p, *run(p, dev, new=False), see_new=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_batch(dtype):
    dev = device()
    g = torch.Generator().manual_seed(1)
    ctx = torch.randint(-1, 40, (3000,), generator=g).tolist()
    p = batch(ctx, hq=2, hkv=2, D=64, B=8, dtype=dtype, seed=2)
    out, lse = (torch.zeros_like(p["q"]).to(dev), torch.zeros((3000, 2), device=dev))
    check(p, *run(p, dev, out=out, lse=lse))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_flat_and_sharp_softmax(scale, dtype):
    dev = device()
    p = batch([2000, 300], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=9, q_scale=scale)
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_slots_past_the_context_may_hold_anything(value, dtype):
    dev = device()
    ctx = [37, 0, 64, 130, 1001]
    p = batch(ctx, hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=4)
    for b, c in enumerate(ctx):
        p["k_pool"][p["table"][b, c // 16], :, c % 16:] = value
        p["v_pool"][p["table"][b, c // 16], :, c % 16:] = value
    for page in set(range(p["k_pool"].shape[0])) - set(p["table"].flatten().tolist()):
        p["k_pool"][page], p["v_pool"][page] = value, value
    check(p, *run(p, dev))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_odd_values_reach_their_row(value, dtype):
    dev = device()
    p = batch([50, 900, 20], hq=4, hkv=2, D=64, B=16, dtype=dtype, seed=4)
    p["v_pool"][p["table"][0, 1], 0, 3, 7] = value
    p["k_pool"][p["table"][1, 20], 1, 3, 7] = value
    p["v"][2, 0] = value
    check(p, *run(p, dev))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_pages_are_left_out(dtype):
    dev = device()
    p = batch([70, 1200, 16, 31, 5], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=2)
    pages = p["k_pool"].shape[0]
    p["table"][0, 2] = -3
    p["table"][1, 0], p["table"][1, 50] = pages, 2 ** 31 - 1
    p["table"][2, 0] = -1      # everything but the new token
    p["table"][3, 1] = pages   # the page that the new token would go to as well
    t = to_gpu(p, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = call(p, t, err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    check(p, out, lse)
    kp, vp = pools_after(p)
    assert torch.equal(bits(t["k_pool"]), bits(kp)) and torch.equal(bits(t["v_pool"]), bits(vp))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_full_table_and_lengths_past_it(dtype):
    """A full page-table row: the token takes part and is not stored (D2F_ERR_BAD_INDEX). A length
    past the row: the sequence is skipped (D2F_ERR_INVALID_ARG)."""
    dev = device()
    p = batch([64, 10], hq=2, hkv=2, D=64, B=16, dtype=dtype, seed=2, spare=0)
    assert p["table"].shape[1] == 4
    t = to_gpu(p, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = call(p, t, err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    check(p, out, lse)
    kp, vp = pools_after(p)
    assert torch.equal(bits(t["k_pool"]), bits(kp)) and torch.equal(bits(t["v_pool"]), bits(vp))
    t["ctx"][0] = 65
    err.zero_()
    out, lse = torch.full_like(out, 7), torch.full_like(lse, 7)
    call(p, t, err=err, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(err) == 1 and bool((out[0] == 7).all()) and bool((lse[0] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_in_a_graph(dtype):
    """A captured step (attention, then ctx_len + 1) replayed: every token sees the ones before,
    with a workspace that other calls use in between."""
    dev = device()
    p = batch([33, 0, 1500, -1], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=11, spare=12)
    t = to_gpu(p, dev)
    n = d2f.token_attn_workspace_size(4, 1512, 4, 2, 128, 16, d2f.BF16 if dtype == BF else d2f.F32)
    m = d2f.logprobs_workspace_size(8, 60000, 4, d2f.F32)
    ws = torch.zeros(max(n, m), dtype=torch.uint8, device=dev)
    out = torch.zeros_like(t["q"])
    lse = torch.zeros(t["q"].shape[:2], device=dev)
    x = torch.randn((8, 60000), device=dev)
    tok = torch.arange(8, dtype=torch.int32, device=dev)
    want = torch.log_softmax(x.double(), -1)[range(8), range(8)]
    call(p, t, workspace=ws, max_ctx=1512)    # (writes the first token's slots; so does the replay)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, t, workspace=ws, max_ctx=1512, out=out, lse=lse)
        t["ctx"].add_((t["ctx"] >= 0).int())
    g = torch.Generator().manual_seed(3)
    for step in range(9):
        for k in ("q", "k", "v"):
            p[k] = torch.randn(p[k].shape, generator=g).to(dtype)
            t[k].copy_(p[k])
        graph.replay()
        lp = d2f.token_logprobs(x, tok, top_k=4, workspace=ws)["logprob"]
        torch.cuda.synchronize()
        assert torch.allclose(lp.double(), want, atol=1e-4)
        check(p, out, lse)
        p["k_pool"], p["v_pool"] = pools_after(p)
        assert torch.equal(bits(t["k_pool"]), bits(p["k_pool"]))
        p["ctx"] = [c + 1 if c >= 0 else c for c in p["ctx"]]
        assert t["ctx"].tolist() == p["ctx"]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeats_and_streams(dtype):
    dev = device()
    p = batch([2000, 70, 5], hq=8, hkv=2, D=128, B=16, dtype=dtype, seed=6)
    t = to_gpu(p, dev)
    first = [x.clone() for x in call(p, t)]
    check(p, *first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({}, dict(stream=side), {}):
        again = call(p, t, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals():
    dev = device()
    p = batch([20, 3], hq=4, hkv=2, D=64, B=16, dtype=BF, seed=1)
    t = to_gpu(p, dev)
    for key, bad in (("q", t["q"].float()), ("k", t["k"][:1]), ("v", t["v"].cpu()),
                     ("k_pool", t["k_pool"][:, :, :8]), ("v_pool", t["v_pool"].transpose(0, 1)),
                     ("table", t["table"].long()), ("ctx", t["ctx"][:1])):
        with pytest.raises((ValueError, TypeError, d2f.D2FError)):
            call(p, dict(t, **{key: bad}))
    with pytest.raises(ValueError):
        d2f.token_attn(t["q"], t["k_pool"], t["v_pool"], t["table"], t["ctx"], block_size=16,
                       max_ctx=20, k_new=t["k"])
    with pytest.raises(d2f.D2FError):
        call(p, t, max_ctx=10 ** 6)
    table = torch.zeros((2, 500), dtype=torch.int32, device=dev)
    with pytest.raises(d2f.D2FError):   # a workspace that is too small
        d2f.token_attn(t["q"], t["k_pool"], t["v_pool"], table, t["ctx"], block_size=16, max_ctx=8000,
                       workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    assert np.isfinite(call(p, t)[1].cpu().numpy()).all()

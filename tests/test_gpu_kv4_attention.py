"""d2f_block_attn_kv4 against float64 attention over the stored values, with elementwise
error bounds (tests/kv4_ref.py)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def problem(ctx, blocks, *, hq, hkv, D, B, dtype, seed, k_exp=0, v_exp=0, extra=2, tail=0,
            k_scale=1.0, v_scale=1.0, q_scale=1.0):
    """CPU inputs of a small layer; `tail` rows behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-c // B) for c in ctx]
    pages = sum(need) + extra
    pool, kv, vv = ref.make_pool(g, pages, hkv, B, D, k_exp, v_exp, k_scale, v_scale)
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(ctx), max(need + [1]) + 1), -1, np.int32)
    for b, m in enumerate(need):
        for i in range(m):
            table[b, i] = order.pop()
    q_start = np.concatenate([[0], np.cumsum([n * B for n in blocks])]).astype(np.int32)
    total = int(q_start[-1]) + tail

    def draw(h, s):
        return (torch.randn((total, h, D), generator=g) * s).to(dtype)
    return dict(q=draw(hq, q_scale), k_win=draw(hkv, k_scale), v_win=draw(hkv, v_scale), pool=pool,
                kv=kv, vv=vv, table=table, ctx=list(ctx), q_start=q_start, B=B, D=D, dtype=dtype,
                k_exp=k_exp, v_exp=v_exp, scale=D ** -0.5)


def run(p, dev, *, max_ctx=None, workspace=None, err=None, stream=None, out=None, lse=None):
    n = np.diff(p["q_start"])
    return d2f.block_attn_kv4(
        p["q"].to(dev), p["k_win"].to(dev), p["v_win"].to(dev), p["pool"].to(dev),
        torch.from_numpy(p["table"]).to(dev),
        torch.tensor(p["ctx"], dtype=torch.int32, device=dev),
        torch.from_numpy(p["q_start"]).to(dev), block_size=p["B"], max_q_per_seq=int(n.max()),
        max_ctx=max(p["ctx"]) if max_ctx is None else max_ctx, k_exp=p["k_exp"],
        v_exp=p["v_exp"], softmax_scale=p["scale"], workspace=workspace, err=err, stream=stream,
        out=out, lse=lse)


def check(p, out, lse):
    o, l, ac, aw, sabs = ref.attention(p["q"], p["k_win"], p["v_win"], p["kv"], p["vv"],
                                       p["table"], p["ctx"], p["q_start"], p["B"], p["scale"])
    n = int(p["q_start"][-1])
    keys = max(p["ctx"]) + int(np.diff(p["q_start"]).max())
    bo, bl = ref.attention_bounds(o, ac, aw, sabs, p["D"], keys, p["dtype"] == torch.bfloat16)
    eo = np.abs(out.double().cpu().numpy() - o)[:n]
    el = np.abs(lse.double().cpu().numpy() - l)[:n]
    assert np.isfinite(eo).all() and np.isfinite(el).all()
    assert (el <= bl[:n]).all(), "lse off by %.3g of its bound" % (el / bl[:n]).max()
    assert (eo <= bo[:n]).all(), "out off by %.3g of its bound" % (eo / bo[:n]).max()


SHAPES = [  # hq, hkv, D, B
    (4, 4, 64, 16), (4, 4, 128, 16), (8, 2, 128, 8), (8, 2, 64, 32), (7, 1, 128, 16),
    (3, 3, 128, 32), (5, 1, 64, 8), (12, 2, 128, 16),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,D,B", SHAPES)
def test_ragged_batch(hq, hkv, D, B, dtype):
    """Contexts of none, one token, a page less one, whole pages, whole tiles and odd ends."""
    dev = device()
    p = problem([0, 1, B - 1, B, 127, 128, 129, 300], [1, 2, 3, 1, 4, 2, 1, 3], hq=hq, hkv=hkv,
                D=D, B=B, dtype=dtype, seed=hq * 1000 + D + B)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(p, out, lse)


@pytest.mark.parametrize("hq,hkv,D,B", SHAPES[::3])
def test_bf16_on_the_cuda_core_path(hq, hkv, D, B, monkeypatch):
    """The switch that forces the CUDA-core kernel (its weights are not rounded: inside the
    tensor-core path's bounds)."""
    dev = device()
    monkeypatch.setenv("D2F_ATTN_PATH", "simt")
    p = problem([0, 1, B, 129, 300], [1, 2, 3, 1, 3], hq=hq, hkv=hkv, D=D, B=B,
                dtype=torch.bfloat16, seed=hq + D + B)
    out, lse = run(p, dev)
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctx,blocks,B", [
    ([2500], [1], 16), ([1024], [3], 16), ([4001, 17], [2, 4], 32), ([1999, 0, 640], [4, 1, 2], 8)])
def test_long_context_split_over_ctas(ctx, blocks, B, dtype):
    dev = device()
    p = problem(ctx, blocks, hq=2, hkv=2, D=128, B=B, dtype=dtype, seed=7, k_exp=1, v_exp=-2,
                v_scale=0.25)
    out, lse = run(p, dev)
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks,hq,hkv", [([9, 5], 2, 1), ([17], 1, 1), ([3, 12], 7, 1),
                                           ([40], 1, 1)])
def test_windows_longer_than_a_tile(blocks, hq, hkv, dtype):
    """Windows of more rows than a row tile and more keys than a key tile."""
    dev = device()
    p = problem([200] * len(blocks), blocks, hq=hq, hkv=hkv, D=128, B=8, dtype=dtype, seed=11)
    out, lse = run(p, dev)
    check(p, out, lse)


@pytest.mark.parametrize("hint", [0, 64, 5000])
def test_max_ctx_is_only_a_hint(hint):
    dev = device()
    p = problem([700, 90], [2, 3], hq=4, hkv=2, D=128, B=16, dtype=torch.bfloat16, seed=3)
    hint = min(hint, p["table"].shape[1] * 16)
    out, lse = run(p, dev, max_ctx=hint)
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_growing_scores_move_the_reference(dtype):
    """Scores that grow along the context by far more than one rescaling step."""
    dev = device()
    p = problem([1200], [2], hq=2, hkv=2, D=128, B=16, dtype=dtype, seed=5)
    # keys along the query, growing page by page
    g = torch.Generator().manual_seed(1)
    u = torch.randn(128, generator=g)
    u = u / u.norm()
    x = np.zeros(p["kv"].shape)
    for i, pg in enumerate(p["table"][0][:75]):
        x[pg] = (u.numpy() * (0.2 * i)) + 0.05 * torch.randn(p["kv"].shape[1:], generator=g).numpy()
    kc, kb, kv = ref.encode(x, 0)
    vc, vb, vv = ref.encode(p["vv"], 0)  # stored values encode to themselves or near them
    p.update(pool=torch.from_numpy(ref.pack_pool(kc, kb, vc, vb)), kv=kv, vv=vv)
    p["q"] = (p["q"] * 0.1 + u * 40.0).to(dtype)
    out, lse = run(p, dev)
    check(p, out, lse)


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 20])
def test_queries_of_any_size(scale):
    """Queries far outside fp16's range (their rows are normalised by a power of two)."""
    dev = device()
    p = problem([333], [2], hq=2, hkv=2, D=128, B=16, dtype=torch.bfloat16, seed=9, q_scale=scale)
    p["scale"] = 128 ** -0.5 / scale
    p["q"][0] *= 2.0 ** -30  # one row much smaller than its neighbours
    out, lse = run(p, dev)
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bytes_past_the_context_may_be_anything(dtype):
    """NaN scales in the slots of the last page past ctx_len and in unused pages."""
    dev = device()
    B, D = 16, 128
    p = problem([37, 130], [2, 1], hq=4, hkv=2, D=D, B=B, dtype=dtype, seed=21)
    clean = run(p, dev)
    pool = p["pool"].clone()
    used = set()
    for b, c in enumerate(p["ctx"]):
        for i in range(-(-c // B)):
            pg = int(p["table"][b][i])
            used.add(pg)
            for o in range(min(B, c - i * B), B):
                pool[pg, :, B * D + o * 8:B * D + o * 8 + 8] = 0x7F
                for grp in range(8):
                    pool[pg, :, B * D + B * D // 16 + grp * B + o] = 0xFF
    for pg in range(pool.shape[0]):
        if pg not in used:
            pool[pg] = 0x7F
    p["pool"] = pool
    out, lse = run(p, dev)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_window_blocks_do_not_reach_a_row(dtype, bad):
    """Infinite or NaN K and V in the last window block: rows of the earlier blocks are those
    of the finite problem, bit by bit."""
    dev = device()
    p = problem([100], [3], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=31)
    clean = run(p, dev)
    p["v_win"][40, 1, 5] = bad
    p["v_win"][33, 0, 127] = -bad
    p["k_win"][45, 0, 3] = bad
    out, lse = run(p, dev)
    assert torch.equal(out[:32], clean[0][:32]) and torch.equal(lse[:32], clean[1][:32])
    # rows that see the value: head group 1's dim 5 is not finite, its other dims are as before
    assert not torch.isfinite(out[32:, 2:, 5]).any()
    keep = [d for d in range(128) if d != 5]
    assert torch.equal(out[32:, 2:][..., keep], clean[0][32:, 2:][..., keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_behind_the_last_sequence_are_left(dtype):
    dev = device()
    p = problem([50, 0], [1, 2], hq=2, hkv=2, D=64, B=16, dtype=dtype, seed=41, tail=32)
    out = torch.full(p["q"].shape, 7.0, dtype=dtype, device=dev)
    lse = torch.full(p["q"].shape[:2], 7.0, device=dev)
    run(p, dev, out=out, lse=lse)
    check(p, out, lse)
    assert (out[48:] == 7).all() and (lse[48:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_pages_are_left_out(dtype):
    dev = device()
    p = problem([200, 64], [1, 1], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=51)
    p["table"][0, 3] = p["pool"].shape[0]
    p["table"][0, 7] = -5
    p["table"][1, 1] = 2 ** 30
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = run(p, dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_inconsistent_sequences_are_reported_and_skipped(dtype):
    dev = device()
    p = problem([64, 64, 64], [1, 1, 1], hq=2, hkv=2, D=64, B=16, dtype=dtype, seed=61)
    p2 = dict(p, ctx=[64, -3, 64])
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full(p["q"].shape, 3.0, dtype=dtype, device=dev)
    lse = torch.zeros(p["q"].shape[:2], device=dev)
    run(p2, dev, err=err, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(err) == 1
    assert (out[16:32] == 3).all()
    good = run(p, dev)
    out[16:32], lse[16:32] = good[0][16:32], good[1][16:32]
    check(p, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_repeats_graphs_and_streams_give_the_same_bits(dtype):
    """The same call again on one workspace, on another stream, and captured and replayed."""
    dev = device()
    p = problem([900, 33, 0, 512], [2, 1, 3, 4], hq=4, hkv=2, D=128, B=16, dtype=dtype, seed=71)
    n = np.diff(p["q_start"])
    dt = d2f.BF16 if dtype == torch.bfloat16 else d2f.F32
    ws = d2f.attn_kv4_workspace(dev, batch=4, total_q=p["q"].shape[0], max_q_per_seq=int(n.max()),
                                max_ctx=900, num_heads_q=4, num_heads_kv=2, head_dim=128,
                                block_size=16, dtype=dt)
    first = run(p, dev, workspace=ws)
    check(p, *first)
    again = run(p, dev, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    q, kw, vw, pool = (p[k].to(dev) for k in ("q", "k_win", "v_win", "pool"))
    table = torch.from_numpy(p["table"]).to(dev)
    ctx = torch.tensor(p["ctx"], dtype=torch.int32, device=dev)
    qs = torch.from_numpy(p["q_start"]).to(dev)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)

    def call(stream=None):
        d2f.block_attn_kv4(q, kw, vw, pool, table, ctx, qs, block_size=16,
                           max_q_per_seq=int(n.max()), max_ctx=900, out=out, lse=lse,
                           workspace=ws, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_no_lse_and_no_context():
    dev = device()
    p = problem([0, 0], [2, 1], hq=4, hkv=4, D=128, B=16, dtype=torch.bfloat16, seed=81)
    out, lse = run(p, dev)
    check(p, out, lse)
    o2, none = d2f.block_attn_kv4(
        p["q"].to(dev), p["k_win"].to(dev), p["v_win"].to(dev), p["pool"].to(dev),
        torch.empty((2, 0), dtype=torch.int32, device=dev),
        torch.zeros(2, dtype=torch.int32, device=dev), torch.from_numpy(p["q_start"]).to(dev),
        block_size=16, max_q_per_seq=32, max_ctx=0, want_lse=False)
    assert none is None and torch.equal(out, o2)

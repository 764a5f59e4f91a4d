"""The softmax weights of d2f_block_attn_kv4 on tensor cores, against float64 with bounds that
leave nothing for lost or coarsely rounded ones."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_common import device
from test_gpu_kv4_attention import problem, run

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -31  # a cached weight's absolute error beside its relative one, of the largest weight


def check(p, out, lse):
    """Elementwise bounds (half steps: fp16 2^-11, bf16 2^-8, fp32 2^-24).

    Score: a float32 sum of D exact products in any order, each addition may truncate (2^-23),
    scaled once. A weight errs by twice that (numerator and normaliser), by 2^-20 of the
    exponential, and by the sums over the keys: 16 keys a step of the matrix product (truncating),
    128 a step of the normaliser. Cached weights round to fp16, window weights to a pair of bf16
    (2^-16). A cached weight that fp16 cannot hold errs by half its smallest number, 2^-25, where
    the largest weight is at least 2^6. The output rounds once."""
    o, l, ac, aw, sabs = ref.attention(p["q"], p["k_win"], p["v_win"], p["kv"], p["vv"],
                                       p["table"], p["ctx"], p["q_start"], p["B"], p["scale"])
    n = int(p["q_start"][-1])
    keys = max(p["ctx"]) + int(np.diff(p["q_start"]).max())
    ds = (p["D"] + 4) * 2.0 ** -23 * sabs
    w = 2 * ds + 2.0 ** -20 + (keys / 16 + 64) * 2.0 ** -23
    err = w[..., None] * (ac + aw) + 2.0 ** -11 * ac + 2.0 ** -16 * aw
    hkv = p["k_win"].shape[1]
    G = p["q"].shape[1] // hkv
    for b, c in enumerate(p["ctx"]):
        lost = np.zeros((hkv, p["D"]))
        for i in range(-(-c // p["B"])):
            lost += np.abs(p["vv"][p["table"][b][i], :, :min(p["B"], c - i * p["B"])]).sum(1)
        err[p["q_start"][b]:p["q_start"][b + 1]] += LOST * np.repeat(lost, G, 0)
    err = err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-30
    eo = np.abs(out.double().cpu().numpy() - o)[:n]
    el = np.abs(lse.double().cpu().numpy() - l)[:n]
    assert np.isfinite(eo).all()
    assert (eo <= err[:n]).all(), "out off by %.3g of its bound" % (eo / err[:n]).max()
    bl = ds + 2.0 ** -18 + (keys / 128 + 64) * 2.0 ** -24
    assert (el <= bl[:n]).all(), "lse off by %.3g of its bound" % (el / bl[:n]).max()


@pytest.mark.parametrize("ctx", [130, 4096, 20000])
@pytest.mark.parametrize("top", [0.0, 40.0, -30.0])
def test_many_small_weights_beside_a_large_one(top, ctx):
    """One key whose V is 0 at 2^top, all others some 2^-27 below it: the output is the small
    weights' alone. (Scores in powers of two: the softmax scale is ln 2, the query 1 in dim 0.)"""
    dev = device()
    D, B = 64, 16
    p = problem([ctx], [1], hq=1, hkv=1, D=D, B=B, dtype=torch.bfloat16, seed=ctx)
    p["scale"] = float(np.log(2.0))
    x = np.zeros(p["kv"].shape)
    x[..., 0] = top - 27
    first = p["table"][0][0]
    x[first, 0, 5, 0] = top
    kc, kb, p["kv"] = ref.encode(x, 0)
    v = np.abs(p["vv"])
    v[first, 0, 5] = 0
    vc, vb, p["vv"] = ref.encode(v, 0)
    p["pool"] = torch.from_numpy(ref.pack_pool(kc, kb, vc, vb))
    assert p["kv"][..., 0].max() - np.median(p["kv"][..., 0]) > 25
    p["q"].zero_()
    p["q"][..., 0] = 1
    p["k_win"].zero_()
    p["k_win"][..., 0] = top - 100
    p["v_win"].zero_()
    check(p, *run(p, dev))


@pytest.mark.parametrize("blocks,hq,hkv,D,B", [([1], 4, 4, 128, 16), ([3, 1, 2], 4, 2, 64, 16),
                                               ([40], 1, 1, 128, 8), ([9, 17], 2, 1, 64, 32),
                                               ([12], 7, 1, 128, 32)])
@pytest.mark.parametrize("v_exp", [0, -3, 2])
def test_window_weights(blocks, hq, hkv, D, B, v_exp):
    """No cached tokens: windows of one and of several key tiles."""
    dev = device()
    p = problem([0] * len(blocks), blocks, hq=hq, hkv=hkv, D=D, B=B, dtype=torch.bfloat16,
                seed=sum(blocks), v_exp=v_exp, v_scale=2.0 ** v_exp)
    check(p, *run(p, dev))


@pytest.mark.parametrize("ctx,blocks,hq,hkv,D,B", [
    ([0, 1, 15, 16, 127, 128, 129, 300], [1, 2, 3, 1, 4, 2, 1, 3], 4, 4, 128, 16),
    ([2500], [1], 2, 2, 128, 16), ([4001, 17], [2, 4], 5, 1, 64, 32),
    ([200, 640], [40, 18], 1, 1, 128, 8), ([900], [9], 7, 1, 64, 16)])
@pytest.mark.parametrize("k_scale", [1.0, 6.0])
def test_cached_and_window_weights(ctx, blocks, hq, hkv, D, B, k_scale):
    """Flat scores, and scores so far apart that the references move."""
    dev = device()
    p = problem(ctx, blocks, hq=hq, hkv=hkv, D=D, B=B, dtype=torch.bfloat16, seed=len(ctx) + D,
                k_scale=k_scale, k_exp=1, v_exp=-2, v_scale=0.25)
    check(p, *run(p, dev))


def test_references_that_rise_many_times():
    """Scores that grow by 2^4 a page over 120 pages, then fall: the last reference is far above
    the first, and the sums before it keep their weight."""
    dev = device()
    D, B, pages = 64, 16, 120
    p = problem([pages * B - 3], [2], hq=2, hkv=1, D=D, B=B, dtype=torch.bfloat16, seed=8)
    p["scale"] = float(np.log(2.0))
    x = np.zeros(p["kv"].shape)
    g = np.random.default_rng(3)
    for i, pg in enumerate(p["table"][0][:pages]):
        x[pg, :, :, 0] = (4 * i if i < 60 else 236 - (i - 60)) + g.uniform(-3, 3, (1, B))
    kc, kb, p["kv"] = ref.encode(x, 0)
    vc, vb, p["vv"] = ref.encode(p["vv"], 0)
    p["pool"] = torch.from_numpy(ref.pack_pool(kc, kb, vc, vb))
    p["q"].zero_()
    p["q"][:, 0, 0] = 1
    p["q"][:, 1, 0] = -0.5
    check(p, *run(p, dev))

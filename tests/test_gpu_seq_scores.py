"""Scores of d2f_prompt_attn and d2f_token_attn that move the softmax's reference, against float64
attention with elementwise bounds (tests/seq_ref.py)."""
import numpy as np
import pytest
import torch

import seq_ref
import test_gpu_prompt_attention as prompts
import test_gpu_token_attention as tokens
from gpu_common import device
from seq_ref import attention, bounds, cached, problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def stairs(p, rise, fall):
    """Scores that grow by about `rise` with every 64 keys, V that shrinks by 2^fall: every step of 64
    keys of the prompt's softmax moves the reference, and the outputs hold what all of them left."""
    at = [torch.arange(n) for n in p["new"]]
    for b, n in enumerate(p["new"]):
        # (the new rows begin a tile of their own, behind the tiles of the cached tokens)
        c, r = p["ctx"][b], int(p["start"][b])
        step = at[b] // 64 + 2 * -(-c // 128)
        p["k"][r:r + n, :, 0] = (rise * p["D"] ** 0.5 * step).to(p["dtype"])[:, None]
        p["v"][r:r + n] *= (2.0 ** (100 - fall * step)).to(p["dtype"])[:, None, None]
        for t in range(c):
            page, off = int(p["table"][b, t // p["B"]]), t % p["B"]
            p["k_pool"][page, :, off, 0] = rise * p["D"] ** 0.5 * (t // 64)
            p["v_pool"][page, :, off] *= 2.0 ** (100 - fall * (t // 64))
    p["q"][..., 0] = 1.0
    return p


def below_float(p, rows):
    """What the keys whose weight is below 2^-125 of the row's largest add to sum p |v|. The softmax of
    parts of the keys (CTAs, warps, lane groups) is put together with one factor 2^(m_part - m) a part,
    which is 0 in float32 below 2^-126, where 64 bits keep it; one power of two is left for the
    reference, which need not be the maximum of the part's own key to the last bit."""
    total, hq, D = p["q"].shape
    G = hq // p["k"].shape[1]
    lost = np.zeros((total, hq, D))
    q, kn, vn = (p[x].double().numpy() for x in "qkv")
    for b, n in enumerate(p["new"]):
        r0 = int(p["start"][b])
        for h in range(hq // G):
            kc, vc = cached(p, b, h)
            for i in (i for i in range(n) if r0 + i in rows):
                end = n if p["mask_block"] == 0 else i + 1
                k = np.concatenate([kc, kn[r0:r0 + end, h]])
                v = np.abs(np.concatenate([vc, vn[r0:r0 + end, h]]))
                for j in range(h * G, h * G + G):
                    s = p["scale"] * (k @ q[r0 + i, j])
                    e = np.exp(s - s.max())
                    lost[r0 + i, j] = np.where(e < 2.0 ** -125, e, 0) / e.sum() @ v
    return lost


def check(p, out, lse, rows):
    o, l, av, sabs, keys = attention(p, rows)
    at = ~np.isnan(l)
    bo, bl = bounds(o, av, sabs, keys, p["D"], p["dtype"] == BF)
    eo = np.abs(out.double().cpu().numpy() - o)[at] / (bo + below_float(p, rows))[at]
    el = np.abs(lse.double().cpu().numpy() - l)[at] / bl[at]
    assert (el <= 1).all(), "lse off by %.3g of its bound" % el.max()
    assert (eo <= 1).all(), "out off by %.3g of its bound" % eo.max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rise,fall", [(9.0, 13), (6.0, 8), (60.0, 0)])
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 128), (7, 1, 128), (2, 1, 64)])
@pytest.mark.parametrize("new,ctx", [([800, 300], [0, 0]), ([150, 40], [640, 700])])
def test_every_step_of_keys_moves_the_reference(new, ctx, hq, hkv, D, rise, fall, dtype):
    """Rises of 2^13, near 2^8 and 2^86 in either half of a tile, many tiles in a row: the weights of
    the tile's first half and the output so far are scaled once each."""
    dev = device()
    p = problem(new, ctx, hq=hq, hkv=hkv, D=D, B=16, dtype=dtype, seed=D + hq, q_scale=0.1)
    p = stairs(p, rise, fall)
    rows = set(range(0, sum(new), 23)) | {63, 64, 127, 128, new[0] - 1, new[0], sum(new) - 1}
    check(p, *prompts.run(p, dev), rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 128), (7, 1, 128), (2, 1, 64)])
def test_single_tokens_whose_keys_move_the_reference(hq, hkv, D, dtype):
    dev = device()
    p = tokens.batch([800, 63, 700], hq=hq, hkv=hkv, D=D, B=16, dtype=dtype, seed=D, q_scale=0.1)
    check(p, *tokens.run(stairs(p, 9.0, 13), dev), {0, 1, 2})


@pytest.mark.parametrize("path", ["", "simt"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("ctx", [0, 40, 2500])
def test_rows_without_a_finite_score_get_zero_whatever_v_holds(ctx, value, dtype, path, monkeypatch):
    """All of a row's scores -infinity: out 0 and lse -infinity, where V holds infinities and NaN too;
    rows of the same tile that see a finite score from another key on keep theirs."""
    if path:
        monkeypatch.setenv("D2F_ATTN_PATH", path)
    dev = device()
    for n, mod in ((150, prompts), (1, tokens)):
        p = problem([n], [ctx], hq=4, hkv=2, D=64, B=16, dtype=dtype, seed=ctx)
        p["mask_block"] = 1 if mod is prompts else 0
        p["q"][..., 0] = 1.0
        for x in ("k", "k_pool"):
            p[x][..., 0] = float("-inf")
        for x in ("v", "v_pool"):
            p[x][:, 0] = value
        out, lse = mod.run(p, dev)
        assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    if ctx == 0:   # a causal prompt whose rows see a finite score from row 70 on
        p = problem([150], [0], hq=4, hkv=2, D=64, B=16, dtype=dtype, seed=1)
        p["q"][..., 0] = 1.0
        p["k"][:70, :, 0] = float("-inf")
        p["v"][100:, 1] = value
        out, lse = prompts.run(p, dev)
        assert bool((out[:70] == 0).all()) and bool((lse[:70] == float("-inf")).all())
        seq_ref.check(p, out, lse, rows=set(range(70, 150)))


@pytest.mark.parametrize("path", ["", "simt"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("low", [3e9, 1e10, 1e20, 2e34])
@pytest.mark.parametrize("D,n,ctx", [(64, 300, 0), (128, 300, 200), (64, 40, 2500)])
@pytest.mark.parametrize("shape", ["low", "high", "rising", "near last", "far last"])
def test_scores_far_from_zero(shape, D, n, ctx, low, dtype, path, monkeypatch):
    """Scores up to 2e33 in magnitude beside rows whose scores are of unit size: a row that sees scores
    far from 0 takes the V of its largest one (the others are further below it than float tells
    apart), whether its reference begins there, gets there or leaves."""
    if path:
        monkeypatch.setenv("D2F_ATTN_PATH", path)
    dev = device()
    p = problem([n], [ctx], hq=4, hkv=2, D=D, B=16, dtype=dtype, seed=n)
    at = np.arange(n)
    far = torch.from_numpy(at % 3 != 0)     # rows that take dim 0 into account
    p["q"][..., 0] = far[:, None].to(dtype)
    p["k_pool"][..., 0] = -low
    k0 = np.full(n, -low)
    best = np.full(n, -1)                   # the key whose V the row takes; -1: none stands out
    near = np.zeros(n, bool)                # rows whose visible scores are of unit size
    if shape in ("low", "high"):
        k0[:] = -low if shape == "low" else low / 4
        k0[5] = -low / 4 if shape == "low" else low
        best[5:] = 5
    elif shape == "rising":                 # one key in 64 above all before it
        for h, j in enumerate(range(5, n, 64)):
            k0[j] = low * 2.0 ** (h - 5)
            best[j:] = j
    elif shape == "near last":
        k0[5] = -low / 4
        best[5:20] = 5
        k0[20:] = 0
        near[20:] = True
    else:
        k0[:20], k0[20] = 0, low
        near[:20] = True
        best[20:] = 20
    p["k"][..., 0] = torch.from_numpy(k0).to(dtype)[:, None]
    out, lse = prompts.run(p, dev)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    # far rows: one weight, rounded to bf16 on the tensor cores, and the output's rounding
    rows = np.flatnonzero((best >= 0) & far.numpy())
    want = p["v"][best[rows]].double().repeat_interleave(2, 1)
    tol = 2.0 ** -8 * (1 + 2.0 ** -7) * 2 if dtype == BF else 2.0 ** -22
    assert bool(((out.cpu().double()[rows] - want).abs() <= tol * want.abs()).all())
    # (float32 products and logarithms: a few roundings of 2^-24; beside them the other dims' part of
    # the score, below 64)
    top = p["scale"] * p["k"][best[rows], :, 0].double().numpy().repeat(2, 1)
    assert np.allclose(lse.cpu().double().numpy()[rows], top, rtol=1e-6, atol=64)
    # rows that leave dim 0 out, and rows over keys of unit size: as if the others scored -250 or less
    p["k"][..., 0] = torch.from_numpy(np.where(k0 < 0, -2000.0 * (D / 64) ** 0.5, 0.0)).to(dtype)[:, None]
    p["k_pool"][..., 0] = -2000.0 * (D / 64) ** 0.5
    rows = set(np.flatnonzero(near | ~far.numpy()).tolist())
    seq_ref.check(p, out, lse, rows=rows)

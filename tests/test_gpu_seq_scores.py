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

"""d2f_token_logprobs against float64 sums.

Bounds. A row's S is a float32 sum of V terms made of partial sums of at most V / 256 + 64
additions a thread and slice, each term off by 2^-21 (argument rounding |x| 2^-24 ln 2 with
|x| <= 64 log2 units where a term matters, 2^-22 of the exponential): ln S is off by at most
2^-17 + (V / 256 + 80) 2^-24. A log probability adds the rounding of two subtractions and of
the logarithm, 3 * 2^-24 of the largest magnitude. The entropy is a quotient of such sums of
terms |t d| <= their absolute sum A = sum p |d| <= H + ln V: off by the same relative error of
A and of ln S.
"""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def check(logits, tokens, k, r, logit_row=None):
    lp, ent, ids, tlp = ref.token_logprobs(logits, tokens, k, logit_row)
    V = logits.shape[1]
    rel = 2.0 ** -17 + (V / 256 + 80) * 2.0 ** -24
    nan = np.isnan(lp)

    def close(got, want, size):
        got = got.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            same = (got == want) | (np.isnan(got) & np.isnan(want))
            ok = same | (np.abs(got - want) <= rel + 3 * 2.0 ** -24 * size)
        assert ok.all(), np.nanmax(np.abs(got - want))
    mag = np.abs(np.nan_to_num(logits.double().numpy(), nan=0, posinf=0, neginf=0)).max() * 2 + 20
    close(r["logprob"], lp, mag)
    assert np.array_equal(np.isnan(r["logprob"].cpu().numpy()), nan)
    A = np.where(nan, 0, np.nan_to_num(ent)) + np.log(V) + 1
    got = r["entropy"].double().cpu().numpy()
    ok = (np.isnan(got) & np.isnan(ent)) | (np.abs(got - ent) <= 2 * rel * A)
    assert ok.all(), np.nanmax(np.abs(got - ent))
    if k:
        assert np.array_equal(r["top_id"].cpu().numpy(), ids)
        close(r["top_logprob"], tlp, mag)


def draw(rows, V, dtype, seed, pad=0, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn((rows, V + pad), generator=g) * sigma).to(dtype)
    tok = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32)
    return buf, tok


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,pad,k", [
    (1, 1, 0, 1), (1, 1, 0, 0), (3, 5, 0, 5), (2, 31, 3, 31), (4, 257, 0, 32), (5, 1000, 0, 5),
    (7, 4099, 5, 20), (3, 20001, 8, 32), (2, 126464, 0, 5), (1, 152064, 0, 20), (40, 6000, 0, 1),
    (700, 3001, 0, 3), (2, 65536, 1, 0)])
def test_random_rows(rows, V, pad, k, dtype):
    dev = device()
    buf, tok = draw(rows, V, dtype, rows * V + k, pad)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    r = d2f.token_logprobs(buf.to(dev)[:, :V], tok.to(dev), top_k=k, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(buf[:, :V], tok.tolist(), k, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 9000, 50001])
def test_ties_and_order(V, dtype):
    """Constant rows, few distinct values, ascending and descending rows, signed zeros."""
    dev = device()
    x = torch.zeros((6, V))
    x[1] = torch.arange(V) % 3
    x[2] = torch.arange(V) / V * 50
    x[3] = 50 - torch.arange(V) / V * 50
    x[4, ::2] = -0.0
    x[5] = float("-inf")
    x[5, V // 2] = 1.0
    x = x.to(dtype)
    tok = torch.tensor([0, V - 1, V - 1, 0, 1, V // 2], dtype=torch.int32)
    r = d2f.token_logprobs(x.to(dev), tok.to(dev), top_k=32)
    check(x, tok.tolist(), 32, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [9, 1000, 126464])
def test_nearly_certain_tokens_keep_their_precision(V, dtype):
    """A token with nearly all the probability: log p = -ln(1 + s) and the entropy are tiny sums
    of positive terms. Each term is off by 2^-22 of the exponential and by its argument's
    rounding (|d| <= 60: 60 * 1.45 * 2^-24), the sums by at most V / 256 + 80 steps of 2^-24, the
    logarithm and quotient by a few: relative to the value, not to 1."""
    dev = device()
    g = torch.Generator().manual_seed(V)
    x = torch.randn((12, V), generator=g)
    tok = torch.randint(0, V, (12,), generator=g)
    x[torch.arange(12), tok] = torch.tensor([8.0, 12, 14, 16, 18, 20, 22, 24, 26, 28, 30, 40])
    x = x.to(dtype)
    r = d2f.token_logprobs(x.to(dev), tok.to(torch.int32).to(dev), top_k=2)
    z = x.double() - x.double().max(-1, keepdim=True).values
    p = z.exp()
    p[torch.arange(12), tok] = 0
    s = p.sum(-1)                                   # (without the token's own 1)
    lp = -torch.log1p(s)
    ent = torch.log1p(s) - (p * z).sum(-1) / (1 + s)
    rel = 2.0 ** -18 + (V / 256 + 90) * 2.0 ** -24
    assert (x.float().argmax(-1) == tok).all()
    assert ((r["logprob"].cpu().double() - lp).abs() <= rel * lp.abs()).all()
    assert ((r["entropy"].cpu().double() - ent).abs() <= 2 * rel * ent).all()
    assert (r["top_id"][:, 0].cpu() == tok).all()
    assert torch.equal(r["top_logprob"][:, 0], r["logprob"])


@pytest.mark.parametrize("V", [50, 30000])
def test_masked_and_broken_logits(V):
    """-inf almost everywhere; all -inf; NaN; +inf: the row's sums are NaN, the list is not."""
    dev = device()
    x = torch.full((5, V), float("-inf"))
    x[0, 3:9] = torch.tensor([1.0, 5.0, 2.0, 2.0, -4.0, 0.0])
    x[2] = torch.randn(V, generator=torch.Generator().manual_seed(1))
    x[2, V - 2] = float("nan")
    x[3] = 0.5
    x[3, 7] = float("inf")
    x[4] = -3e38
    tok = torch.tensor([4, 0, 1, 2, 9], dtype=torch.int32)
    r = d2f.token_logprobs(x.to(dev), tok.to(dev), top_k=8)
    lp, ent, ids, tlp = ref.token_logprobs(x, tok.tolist(), 8)
    got = {k: v.cpu() for k, v in r.items()}
    assert np.array_equal(got["top_id"].numpy(), ids)
    for row in (1, 2, 3):
        assert torch.isnan(got["logprob"][row]) and torch.isnan(got["entropy"][row])
    for row in (0, 4):
        assert abs(float(got["logprob"][row]) - lp[row]) < 1e-5 * max(1, abs(lp[row]))
        assert abs(float(got["entropy"][row]) - ent[row]) < 1e-4
    assert torch.isneginf(got["top_logprob"][0, 6:]).all()
    # a token of probability zero
    r = d2f.token_logprobs(x.to(dev)[:1], torch.tensor([0], dtype=torch.int32, device=dev))
    assert torch.isneginf(r["logprob"]).all()


@pytest.mark.parametrize("dtype,V,pad", [(torch.bfloat16, 9000, 0), (torch.bfloat16, 9001, 4),
                                         (torch.float32, 9003, 0), (torch.float32, 40, 0)])
def test_alternatives_beside_nan_are_the_lowest_indices(dtype, V, pad):
    """Rows of NaN and -inf: the -inf logits are alternatives in order of index, whatever
    shares the vocabulary pass gives a thread; fewer of them than k leave -1."""
    dev = device()
    g = torch.Generator().manual_seed(3)
    x = torch.full((6, V + pad), float("-inf"))
    x[0, :V][torch.arange(V) % 2048 < 96] = float("nan")  # whole threads without a number
    x[1, :V - 3] = float("nan")
    x[2, :V] = torch.where(torch.rand(V, generator=g) < 0.9, float("nan"), float("-inf"))
    x[3, :V] = float("nan")
    x[4, 7:V] = float("nan")
    x[4, 20] = 1.5
    x[5, :V] = torch.where(torch.rand(V, generator=g) < 0.5, float("nan"), float("-inf"))
    x[5, V - 1] = -2.0
    x = x.to(dtype)
    k = 10
    r = d2f.token_logprobs(x.to(dev)[:, :V], torch.arange(6, dtype=torch.int32, device=dev), top_k=k)
    for row in range(6):
        v = x[row, :V].float().numpy()
        real = np.nonzero(~np.isnan(v))[0]
        want = real[np.argsort(-v[real], kind="stable")][:k].tolist()
        assert r["top_id"][row].tolist() == want + [-1] * (k - len(want))
    assert torch.isnan(r["logprob"]).all() and torch.isnan(r["entropy"]).all()


def test_rows_without_a_token_and_bad_indices():
    dev = device()
    V = 8000
    buf, tok = draw(6, V, torch.bfloat16, 3)
    tok[1], tok[4] = -1, -100
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    r = d2f.token_logprobs(buf.to(dev), tok.to(dev), top_k=4, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(buf, tok.tolist(), 4, r)
    tok[0] = V
    rows = torch.tensor([0, 0, 6, 3, 4, -1], dtype=torch.int32)
    r = d2f.token_logprobs(buf.to(dev), tok.to(dev), top_k=4, logit_row=rows.to(dev), err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    t = tok.tolist()
    t[0] = t[2] = t[5] = -1
    check(buf, t, 4, r, [0, 0, 0, 3, 4, 0])


def test_logit_rows_shift_and_repeat():
    dev = device()
    buf, tok = draw(9, 5001, torch.float32, 4)
    rows = torch.tensor([8, 0, 0, 3, 7, 8], dtype=torch.int32)
    r = d2f.token_logprobs(buf.to(dev), tok[:6].to(dev), top_k=6, logit_row=rows.to(dev))
    check(buf, tok[:6].tolist(), 6, r, rows.tolist())


@pytest.mark.parametrize("rows", [3, 700])
def test_repeats_graphs_and_streams_give_the_same_bits(rows):
    dev = device()
    V = 20000
    buf, tok = draw(rows, V, torch.bfloat16, 5)
    x, t = buf.to(dev), tok.to(dev)
    ws = d2f.logprobs_workspace(dev, n=rows, vocab=V, top_k=7, dtype=d2f.BF16)
    a = d2f.token_logprobs(x, t, top_k=7, workspace=ws)
    b = d2f.token_logprobs(x, t, top_k=7, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = d2f.token_logprobs(x, t, top_k=7, workspace=ws, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = d2f.token_logprobs(x, t, top_k=7, workspace=ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) and torch.equal(a[k], d[k])

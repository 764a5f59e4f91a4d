"""Plain 64-bit attention of packed prompts and of single tokens over a paged cache (NumPy on the
CPU, nothing of the library), the problems that the GPU tests give it, and their error bounds.

Half-step rounding errors, relative to the value: bf16 2^-8, fp32 2^-24.
"""
import numpy as np
import torch


def problem(new, ctx, *, hq, hkv, D, B, dtype, seed, mask_block=1, tail=0, extra=2, q_scale=1.0,
            spare=1):
    """CPU inputs of a batch: `new` rows a request behind `ctx` cached tokens, `tail` rows behind
    the last request, `extra` pages that nobody uses, room for `spare` more tokens a sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(c, 0) + spare) // B) for c in ctx]
    pages = sum(need) + extra

    def draw(*shape, s=1.0):
        return (torch.randn(shape, generator=g) * s).to(dtype)
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(ctx), max(need + [1])), -1, np.int32)
    for b, m in enumerate(need):
        table[b, :m] = order[:m]
        order = order[m:]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(start[-1]) + tail
    return dict(q=draw(total, hq, D, s=q_scale), k=draw(total, hkv, D), v=draw(total, hkv, D),
                k_pool=draw(pages, hkv, B, D), v_pool=draw(pages, hkv, B, D), table=table,
                ctx=list(ctx), new=list(new), start=start, B=B, D=D, dtype=dtype,
                mask_block=mask_block, scale=D ** -0.5)


def cached(p, b, h, n_pages=None):
    """K and V float64 [tokens, D] of a sequence's cached tokens; a page out of range is left out."""
    k, v = [np.zeros((0, p["D"]))], [np.zeros((0, p["D"]))]
    for i in range(-(-p["ctx"][b] // p["B"])):
        page, m = int(p["table"][b, i]), min(p["B"], p["ctx"][b] - i * p["B"])
        if 0 <= page < p["k_pool"].shape[0]:
            k.append(p["k_pool"][page, h, :m].double().numpy())
            v.append(p["v_pool"][page, h, :m].double().numpy())
    return np.concatenate(k), np.concatenate(v)


def attention(p, rows=None, see_new=True):
    """out, lse, sum p |v|, the largest scale sum |q k| of a row and its number of keys, float64 per
    (row, head); NaN in rows that no request owns or that `rows` (a set) leaves out."""
    total, hq, D = p["q"].shape
    hkv = p["k"].shape[1]
    G = hq // hkv
    q, kn, vn = (p[x].double().numpy() for x in "qkv")
    out, av = np.full((total, hq, D), np.nan), np.zeros((total, hq, D))
    lse, sabs, keys = (np.full((total, hq), x) for x in (np.nan, 0.0, 0))
    mb = p["mask_block"]
    for b, n in enumerate(p["new"]):
        r0 = int(p["start"][b])
        mine = [i for i in range(n) if rows is None or r0 + i in rows]
        if p["ctx"][b] < 0 or not mine:
            continue
        for h in range(hkv):
            kc, vc = cached(p, b, h)
            for i in mine:
                end = n if mb == 0 else min(n, (i // mb + 1) * mb)
                end = end if see_new else 0
                k = np.concatenate([kc, kn[r0:r0 + end, h]])
                v = np.concatenate([vc, vn[r0:r0 + end, h]])
                for j in range(h * G, (h + 1) * G):
                    r = (r0 + i, j)
                    keys[r] = len(k)
                    if len(k) == 0:
                        out[r], lse[r] = 0.0, -np.inf
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = p["scale"] * (k @ q[r])
                        m = s.max()
                        e = np.exp(s - m)
                        l = e.sum()
                        out[r] = (e / l) @ v
                        av[r] = (e / l) @ np.abs(v)
                        lse[r] = m + np.log(l)
                        sabs[r] = (p["scale"] * (np.abs(k) @ np.abs(q[r]))).max()
    return out, lse, av, sabs, keys


def bounds(out, av, sabs, keys, D, bf16):
    """Elementwise bounds on |out error| and |lse error|.

    A score is a float32 sum of D exact products whose order is free and whose additions may
    truncate (one step, 2^-23 each), scaled once: |ds| <= (D + 4) 2^-23 scale sum |q k|. A weight
    then errs by 2 |ds| (numerator and normaliser) plus 2^-20 for the exponential (the argument's
    rounding and 2^-22 of the instruction) and the float32 sums over its keys, and again as much
    for the composition of parts. With bf16 operands the weights of the product with V are
    rounded to bf16 (2^-8) and the output rounds once."""
    ds = (D + 4) * 2.0 ** -23 * sabs
    w = 2 * ds + 2.0 ** -19 + keys * 2.0 ** -23
    err = w[..., None] * av + 1e-30
    if bf16:
        err = err + 2.0 ** -8 * av
    err = err * (1 + 2.0 ** -8) + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(out)
    return err, ds + 2.0 ** -18 + keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(ds)


def check(p, out, lse, rows=None, see_new=True):
    """Compare with the 64-bit form, elementwise; infinities and NaN have to be the same ones."""
    o, l, av, sabs, keys = attention(p, rows, see_new)
    at = ~np.isnan(l) | (keys > 0)
    with np.errstate(invalid="ignore", over="ignore"):
        bo, bl = bounds(o, av, sabs, keys, p["D"], p["dtype"] == torch.bfloat16)
        eo = np.abs(out.double().cpu().numpy() - o)[at]
        el = np.abs(lse.double().cpu().numpy() - l)[at]
    got_o, got_l = out.double().cpu().numpy()[at], lse.double().cpu().numpy()[at]
    fo, fl = np.isfinite(o[at]), np.isfinite(l[at])
    assert np.array_equal(np.isnan(got_o), np.isnan(o[at])), "NaN elsewhere"
    assert np.array_equal(got_o[~fo & ~np.isnan(o[at])], o[at][~fo & ~np.isnan(o[at])])
    assert np.array_equal(got_l[~fl], l[at][~fl], equal_nan=True)
    assert np.isfinite(got_o[fo]).all() and np.isfinite(got_l[fl]).all()
    assert (el[fl] <= bl[at][fl]).all(), "lse off by %.3g of its bound" % (el[fl] / bl[at][fl]).max()
    assert (eo[fo] <= bo[at][fo]).all(), "out off by %.3g of its bound" % (eo[fo] / bo[at][fo]).max()

"""Plain 64-bit forms of the 4-bit cache, its attention, the page map and the token log
probabilities (NumPy / torch on the CPU, nothing of the library), and the error bounds the
GPU tests use.

Half-step rounding errors, relative to the value: fp16 2^-11, bf16 2^-8, fp32 2^-24.
"""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table():
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = np.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return out


E4M3 = e4m3_table()


def _nearest(x, levels):
    """Index of the level nearest to x >= 0 (ties to the even index; past the top: the top)."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo = np.searchsorted(mid, x, side="left")
    hi = np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def encode(x, exp):
    """x [..., D] (float64 array) -> codes, scale bits, values; a group of 16 shares a scale.

    The definition's divisions are float32 ones: they are made here in float32 too."""
    y = (x.reshape(x.shape[:-1] + (-1, 16)) * 2.0 ** -exp).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(y).max(-1)
        s_in = amax / np.float32(6.0)
        bits = _nearest(np.where(np.isnan(s_in), 0, s_in).astype(np.float64), E4M3[:127])
        bits = np.where(np.isnan(s_in), 127, bits)
        s = E4M3[bits][..., None]
        r = np.where(s > 0, y / np.where(s > 0, s, 1.0).astype(np.float32), 0.0)
        mag = np.abs(r).astype(np.float64)
        codes = np.where(np.isnan(mag), 7, _nearest(np.nan_to_num(mag, nan=0.0, posinf=1e30), E2M1))
        val = E2M1[codes] * s * np.where(np.signbit(r), -1.0, 1.0) * 2.0 ** exp
    codes = codes + 8 * (np.signbit(r) & ~np.isnan(r))
    return codes.reshape(x.shape).astype(np.uint8), bits.astype(np.uint8), val.reshape(x.shape)


def page_tile(k_codes, k_bits, v_codes, v_bits):
    """One page and head: codes [B, D], scale bits [B, D / 16] -> uint8 [page bytes]."""
    B, D = k_codes.shape
    tile = np.zeros(B * D * 9 // 8, np.uint8)
    for t in range(B):
        for d in range(D):
            tile[(d // 32) * B * 16 + t * 16 + (d % 32) // 2] |= k_codes[t, d] << (4 * (d % 2))
            tile[B * D // 2 + d * (B // 2) + t // 2] |= v_codes[t, d] << (4 * (t % 2))
    tile[B * D:B * D + B * D // 16] = k_bits.reshape(-1)
    tile[B * D + B * D // 16:] = v_bits.T.reshape(-1)
    return tile


def tile_values(tile, B, D, k_exp, v_exp):
    """uint8 [page bytes] -> K, V float64 [B, D]."""
    t, d = np.meshgrid(np.arange(B), np.arange(D), indexing="ij")
    kb = tile[(d // 32) * B * 16 + t * 16 + (d % 32) // 2] >> (4 * (d % 2)) & 15
    vb = tile[B * D // 2 + d * (B // 2) + t // 2] >> (4 * (t % 2)) & 15
    ks = E4M3[tile[B * D + t * (D // 16) + d // 16]]
    vs = E4M3[tile[B * D + B * D // 16 + (d // 16) * B + t]]

    def val(c, s, e):
        with np.errstate(invalid="ignore"):
            return E2M1[c & 7] * np.where(c & 8, -1.0, 1.0) * s * 2.0 ** e
    return val(kb, ks, k_exp), val(vb, vs, v_exp)


def pack_pool(kc, kb, vc, vb):
    """Codes [pages, hkv, B, D] and scale bits [pages, hkv, B, D / 16] -> uint8 pool."""
    n, hkv, B, D = kc.shape
    pool = np.zeros((n, hkv, B * D * 9 // 8), np.uint8)
    k = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, hkv, B, D // 32, 16)
    pool[..., :B * D // 2] = k.transpose(0, 1, 3, 2, 4).reshape(n, hkv, -1)
    v = (vc[:, :, 0::2] | (vc[:, :, 1::2] << 4)).transpose(0, 1, 3, 2)
    pool[..., B * D // 2:B * D] = v.reshape(n, hkv, -1)
    pool[..., B * D:B * D + B * D // 16] = kb.reshape(n, hkv, -1)
    pool[..., B * D + B * D // 16:] = vb.transpose(0, 1, 3, 2).reshape(n, hkv, -1)
    return pool


def make_pool(gen, num_pages, hkv, B, D, k_exp=0, v_exp=0, k_scale=1.0, v_scale=1.0):
    """A random pool (uint8 tensor) and its K, V values float64 [pages, hkv, B, D]."""
    def draw(s):
        x = torch.randn((num_pages, hkv, B, D), generator=gen, dtype=torch.float64) * s
        return x.to(torch.bfloat16).double().numpy()
    kc, kb, kv = encode(draw(k_scale), k_exp)
    vc, vb, vv = encode(draw(v_scale), v_exp)
    return torch.from_numpy(pack_pool(kc, kb, vc, vb)), kv, vv


def attention(q, k_win, v_win, kv, vv, page_table, ctx, q_start, B, scale):
    """Attention in float64: out, lse and the terms of the error bound.

    kv, vv: values [pages, hkv, B, D]. Pages outside the pool are left out. Returns out, lse,
    ac = sum over cached keys of p |v|, aw = over window keys (as out), and sabs [rows, Hq] =
    the largest scale * sum |q| |k| over the row's keys."""
    total, hq, D = q.shape
    hkv = k_win.shape[1]
    G = hq // hkv
    q, k_win, v_win = (x.double().numpy() for x in (q, k_win, v_win))
    out = np.zeros((total, hq, D))
    ac, aw = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((total, hq), -np.inf)
    sabs = np.zeros((total, hq))
    for b in range(len(ctx)):
        r0, r1 = q_start[b], q_start[b + 1]
        C = ctx[b]
        pages = [int(p) for p in page_table[b][:-(-C // B)]]
        for h in range(hkv):
            ks, vs = [np.zeros((0, D))], [np.zeros((0, D))]
            for i, p in enumerate(pages):
                m = min(B, C - i * B)
                if 0 <= p < kv.shape[0]:
                    ks.append(kv[p, h, :m])
                    vs.append(vv[p, h, :m])
            kc, vc = np.concatenate(ks), np.concatenate(vs)
            for r in range(r0, r1):
                end = r0 + ((r - r0) // B + 1) * B
                k = np.concatenate([kc, k_win[r0:end, h]])
                v = np.concatenate([vc, v_win[r0:end, h]])
                for j in range(h * G, (h + 1) * G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (k @ q[r, j])
                        m = s.max()
                        p = np.exp(s - m)
                        l = p.sum()
                        p /= l
                        out[r, j] = p @ v
                        ac[r, j] = p[:len(kc)] @ np.abs(vc)
                        aw[r, j] = p[len(kc):] @ np.abs(v[len(kc):])
                        lse[r, j] = m + math.log(l) if l > 0 else np.nan
                        sabs[r, j] = (scale * (np.abs(k) @ np.abs(q[r, j]))).max()
    return out, lse, ac, aw, sabs


def attention_bounds(out, ac, aw, sabs, D, n_keys, bf16):
    """Elementwise bounds on |out error| and |lse error|.

    A score is a float32 sum of D exact products whose order is free and whose additions may
    truncate (one step, 2^-23 each), scaled once: |ds| <= (D + 4) 2^-23 scale sum |q k|. A
    weight then errs by 2 |ds| (numerator and normaliser) plus 2^-20 for the exponential
    (argument rounding at |x| <= 8 beside the reference, 2^-22 of the instruction) and the
    float32 sums over n_keys. On tensor cores the weights of the P.V product are rounded:
    cached keys to fp16 (2^-11), window keys to bf16 (2^-8). The output rounds once."""
    ds = (D + 4) * 2.0 ** -23 * sabs
    w = 2 * ds + 2.0 ** -20 + n_keys * 2.0 ** -23
    a = ac + aw
    err = w[..., None] * a + 1e-30
    if bf16:
        err = err + 2.0 ** -11 * ac + 2.0 ** -8 * aw + 2.0 ** -24
    err = err * (1 + 2.0 ** -8) + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(out)
    return err, ds + 2.0 ** -18 + n_keys * 2.0 ** -24


def page_map(num_new, ctx, table, free_pages, free_count, B, capacity, max_append):
    """The page map, request by request. Returns a dict of lists / arrays."""
    table = np.array(table).copy()
    free = [int(x) for x in free_pages[:free_count]]
    budget = min(free_count, max_append)
    used, row = 0, 0
    r = dict(ctx_len=[], admitted=[], row_start=[0], slot=[-1] * capacity, src=[], dst=[], rows=[])
    wanted = 0
    for b, n in enumerate(num_new):
        need = -(-n // B)
        fits = ctx[b] // B + need <= table.shape[1]
        if fits:
            wanted += need
        ok = fits and wanted <= budget
        if ok:
            for i in range(need):
                page = free.pop()
                used += 1
                table[b, ctx[b] // B + i] = page
                m = min(B, n - i * B)
                r["src"].append(row + i * B)
                r["dst"].append(page)
                r["rows"].append(m)
                for t in range(m):
                    r["slot"][row + i * B + t] = page * B + t
        row += n
        r["admitted"].append(int(ok))
        r["ctx_len"].append(ctx[b] + (n if ok else 0))
        r["row_start"].append(row)
    r["table"], r["n_append"], r["free_count"] = table, used, free_count - used
    pad = max_append - used
    r["src"] += [-1] * pad
    r["dst"] += [-1] * pad
    r["rows"] += [0] * pad
    return r


def token_logprobs(logits, tokens, k, logit_row=None):
    """float64 log probability, entropy, top ids and their log probabilities per row."""
    n = len(tokens)
    lp, ent = np.zeros(n), np.zeros(n)
    ids, tlp = np.full((n, k), -1), np.zeros((n, k))
    for r, t in enumerate(tokens):
        if t < 0:
            continue
        x = logits[r if logit_row is None else logit_row[r]].double().numpy()
        with np.errstate(invalid="ignore", divide="ignore"):
            m = x.max()
            z = x - m
            S = np.exp(z).sum()
            lp[r] = z[t] - math.log(S) if S > 0 else np.nan
            ent[r] = math.log(S) - np.where(z == -np.inf, 0.0, np.exp(z) * z).sum() / S \
                if S > 0 else np.nan
            o = np.argsort(np.where(np.isnan(x), np.inf, -(x + 0.0)), kind="stable")[:k]
        ids[r] = o
        tlp[r] = z[o] - math.log(S) if S > 0 else np.nan
    return lp, ent, ids, tlp

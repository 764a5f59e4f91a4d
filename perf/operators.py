"""Cases that measure the 4-bit paged cache (its page map, its writing and reading back, the
attention over it) and the log probabilities of committed tokens.

Shapes are those of this repository's workloads (LLaDA-8B-shaped layers: 32 heads, head_dim 128,
vocabulary 126,464; Dream-7B-shaped: 28 query heads on 4 KV heads, vocabulary 152,064; blocks of
8, 16 or 32 tokens; contexts up to 32,768) or generic. `run` computes an operator in plain torch
operations while `own` is false and calls block_causal_kv_gb300.d2f while it is true.

The cache page of one KV head (D = head_dim, B = block_size; 16 elements along the head
dimension share one e4m3 scale, an element is one e2m1 code, low nibble first):
  K codes   [D / 32][B][16]  byte i of chunk c of token t: dims 32c + 2i, 32c + 2i + 1
  V codes   [D][B / 2]       byte i of dim d: tokens 2i, 2i + 1
  K scales  [B][D / 16]
  V scales  [D / 16][B]
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the smallest layer of this repository's workloads, float32: one short request
        dict(name="attn_tiny", op="attention", dtype="f32", batch=1, hq=4, hkv=4, d=64, block=16,
             ctx=64, ctx_min=64, blocks=2, blocks_min=2, k_exp=0, v_exp=0, layout=1),
        # one request decoding with a short context: latency of a single layer
        dict(name="attn_llada", op="attention", dtype="bf16", batch=1, hq=32, hkv=32, d=128,
             block=16, ctx=1024, ctx_min=1024, blocks=3, blocks_min=3, k_exp=0, v_exp=-2, layout=2),
        # a served batch: contexts and windows of every length, partly filled last pages
        dict(name="attn_ragged", op="attention", dtype="bf16", batch=16, hq=32, hkv=32, d=128,
             block=16, ctx=4096, ctx_min=251, blocks=3, blocks_min=1, k_exp=0, v_exp=-2, layout=3),
        # grouped heads: 7 query heads share a KV head, so the products bound it
        dict(name="attn_dream", op="attention", dtype="bf16", batch=8, hq=28, hkv=4, d=128,
             block=16, ctx=8192, ctx_min=8192, blocks=3, blocks_min=3, k_exp=0, v_exp=0, layout=4),
        # the longest contexts: the cache read bounds it
        dict(name="attn_long", op="attention", dtype="bf16", batch=4, hq=32, hkv=32, d=128,
             block=16, ctx=32768, ctx_min=32768, blocks=4, blocks_min=4, k_exp=0, v_exp=0,
             layout=5),
        # one decode step's finished blocks, one a request
        dict(name="cache_step", op="cache", dtype="bf16", batch=8, hkv=4, d=128, block=16,
             tokens=16, tokens_min=16, k_exp=0, v_exp=-2, layout=6),
        # the prompts of a served batch, of every length
        dict(name="cache_prompts", op="cache", dtype="bf16", batch=16, hkv=32, d=128, block=16,
             tokens=4096, tokens_min=251, k_exp=1, v_exp=-3, layout=7),
        # a few requests enter a batch
        dict(name="pages_few", op="pages", batch=16, block=16, new=512, new_min=1, cached=0,
             short=0, layout=8),
        # a full queue of requests, some with a cached prefix, more than the free pages hold
        dict(name="pages_many", op="pages", batch=1024, block=16, new=4096, new_min=0, cached=64,
             short=700, layout=9),
        # one request's window, float32 logits of a small vocabulary
        dict(name="logprobs_tiny", op="logprobs", dtype="f32", rows=32, vocab=1000, pad=0, top=5,
             given=0.7, layout=10),
        # one request's window, every position committed
        dict(name="logprobs_llada", op="logprobs", dtype="bf16", rows=48, vocab=126464, pad=0,
             top=5, given=1.0, layout=11),
        # a served batch's windows, half of the positions still masked, twenty alternatives
        dict(name="logprobs_dream", op="logprobs", dtype="bf16", rows=384, vocab=152064, pad=0,
             top=20, given=0.5, layout=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_attention(rng):
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hkv = rng.choice([(32, 32), (28, 4), (4, 4), (8, 2), (32, 8), (5, 1)])
    ctx = _log_int(rng, 1, 32768 if dtype == "bf16" else 2048)
    blocks = rng.randint(1, 4)
    return dict(op="attention", dtype=dtype, batch=_log_int(rng, 1, 16), hq=hq, hkv=hkv,
                d=rng.choice([64, 128, 128]), block=rng.choice([8, 16, 16, 32]), ctx=ctx,
                ctx_min=rng.choice([ctx, rng.randint(0, ctx)]), blocks=blocks,
                blocks_min=rng.randint(1, blocks), k_exp=rng.randint(-2, 2),
                v_exp=rng.randint(-4, 1), layout=rng.randrange(1 << 30))


def _draw_cache(rng):
    tokens = _log_int(rng, 1, 4096)
    return dict(op="cache", dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_log_int(rng, 1, 16),
                hkv=rng.choice([1, 2, 4, 8, 32]), d=rng.choice([64, 128]),
                block=rng.choice([8, 16, 32]), tokens=tokens, tokens_min=rng.randint(1, tokens),
                k_exp=rng.randint(-2, 2), v_exp=rng.randint(-4, 1),
                layout=rng.randrange(1 << 30))


def _draw_pages(rng):
    new = _log_int(rng, 1, 4096)
    return dict(op="pages", batch=_log_int(rng, 1, 1024), block=rng.choice([8, 16, 32]), new=new,
                new_min=rng.randint(0, new), cached=rng.choice([0, 0, rng.randint(1, 64)]),
                short=rng.choice([0, 0, rng.randint(1, 999)]), layout=rng.randrange(1 << 30))


def _draw_logprobs(rng):
    return dict(op="logprobs", dtype=rng.choice(["bf16", "bf16", "f32"]),
                rows=_log_int(rng, 1, 384), vocab=_log_int(rng, 1000, 160000),
                pad=rng.choice([0, 0, rng.randint(1, 64)]), top=rng.choice([0, 1, 5, 20, 32]),
                given=rng.choice([1.0, round(rng.uniform(0.2, 1.0), 2)]),
                layout=rng.randrange(1 << 30))


def draw(rng):
    make = rng.choice([_draw_attention, _draw_attention, _draw_cache, _draw_pages, _draw_logprobs])
    bounds = [work(c) for c in listed()]
    most = {k: max(b[k] for b in bounds) for k in ("bytes", "flops")}
    while True:
        case = make(rng)
        w = work(case)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


# ---------------------------------------------------------------------------
# layouts that a case stands for (host integers)
# ---------------------------------------------------------------------------
def _spread(rng, n, lo, hi):
    """n lengths of [lo, hi], both ends among them where n allows."""
    out = [rng.randint(lo, hi) for _ in range(n)]
    out[0] = hi
    if n > 1:
        out[-1] = lo
    rng.shuffle(out)
    return out


def _attention_layout(c):
    rng = random.Random(c["layout"])
    ctx = _spread(rng, c["batch"], c["ctx_min"], c["ctx"])
    win = [w * c["block"] for w in _spread(rng, c["batch"], c["blocks_min"], c["blocks"])]
    return ctx, win


def _cache_layout(c):
    return _spread(random.Random(c["layout"]), c["batch"], c["tokens_min"], c["tokens"])


def _pages_layout(c):
    """New tokens and cached pages of each request, and the free pages: `short` thousandths of
    what the requests need, or with 0 a few more than that."""
    rng = random.Random(c["layout"])
    new = _spread(rng, c["batch"], c["new_min"], c["new"])
    cached = [rng.randint(0, c["cached"]) if c["cached"] else 0 for _ in new]
    need = sum(-(-n // c["block"]) for n in new)
    free = need + 7 if c["short"] == 0 else need * c["short"] // 1000
    return new, cached, free


def _admit(new, block, free):
    """Requests admitted: the longest prefix whose pages fit the free list."""
    pages = 0
    for i, n in enumerate(new):
        pages += -(-n // block)
        if pages > free:
            return i
    return len(new)


def _given_rows(c):
    rng = random.Random(c["layout"])
    return [rng.random() < c["given"] for _ in range(c["rows"])]


def work(case):
    c = case
    if c["op"] == "attention":
        ctx, win = _attention_layout(c)
        e = 2 if c["dtype"] == "bf16" else 4
        rows, toks = sum(win), sum(ctx)
        cache = toks * c["hkv"] * 2 * (c["d"] // 2 + c["d"] // 16)
        pages = sum(-(-t // c["block"]) for t in ctx)
        data = rows * (2 * c["hq"] + 2 * c["hkv"]) * c["d"] * e + rows * c["hq"] * 4
        seen = sum(n * t + sum(c["block"] * (j + 1) * c["block"] for j in range(n // c["block"]))
                   for t, n in zip(ctx, win))
        return {"bytes": cache + data + 4 * (pages + 2 * c["batch"] + 1),
                "flops": 4 * c["d"] * c["hq"] * seen}
    if c["op"] == "cache":
        e = 2 if c["dtype"] == "bf16" else 4
        lens = _cache_layout(c)
        t, n = sum(lens), sum(-(-x // c["block"]) for x in lens)
        kv = 2 * c["hkv"] * c["d"]
        # written whole pages, read back token by token
        return {"bytes": t * kv * e * 2 + (t + n * c["block"]) * kv * 9 // 16 + 8 * t + 12 * n,
                "flops": 8 * t * kv}
    if c["op"] == "pages":
        new, _, free = _pages_layout(c)
        k = _admit(new, c["block"], free)
        pages = sum(-(-n // c["block"]) for n in new[:k])
        entries = sum(-(-n // c["block"]) for n in new)
        return {"bytes": 8 * sum(new) + 8 * pages + 12 * entries + 17 * len(new) + 16,
                "flops": 4 * sum(new)}
    rows = sum(_given_rows(c))
    e = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": rows * (c["vocab"] * e + 8 + 8 * c["top"]) + 4 * c["rows"],
            "flops": 6 * rows * c["vocab"]}


# ---------------------------------------------------------------------------
# the 4-bit format in plain torch
# ---------------------------------------------------------------------------
def _encode(x, exp):
    """x [..., D] float32 -> (codes uint8 [..., D], scales e4m3 bits uint8 [..., D / 16])."""
    y = (x * 2.0 ** -exp).unflatten(-1, (-1, 16))
    s8 = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    r = torch.where(s == 0, torch.zeros_like(y), y / s)
    m = r.abs()
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte()
            + (m > 2.5).byte() + (m >= 3.5).byte() + (m > 5.0).byte())
    code = code + 8 * (r < 0).byte()
    return code.flatten(-2), s8.view(torch.uint8)


def _pack_pages(kc, ks, vc, vs):
    """Codes [n, B, H, D] and scales [n, B, H, D / 16] of n pages -> uint8 [n, H, page bytes]."""
    n, B, H, D = kc.shape
    k = kc[..., 0::2] | (kc[..., 1::2] << 4)                       # [n, B, H, D / 2]
    k = k.view(n, B, H, D // 32, 16).permute(0, 2, 3, 1, 4).reshape(n, H, -1)
    v = (vc[:, 0::2] | (vc[:, 1::2] << 4)).permute(0, 2, 3, 1).reshape(n, H, -1)
    return torch.cat([k, v, ks.permute(0, 2, 1, 3).reshape(n, H, -1),
                      vs.permute(0, 2, 3, 1).reshape(n, H, -1)], dim=2)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decode_pages(tiles, B, D, k_exp, v_exp):
    """uint8 [n, H, page bytes] -> K, V float32 [H, n * B, D]."""
    n, H, _ = tiles.shape
    lut = torch.tensor(_E2M1, dtype=torch.float32, device=tiles.device)
    half = B * D // 2
    ns = B * D // 16

    def nibbles(x):                                                # [...] -> [..., 2 * last]
        return lut[torch.stack([x & 15, x >> 4], dim=-1).flatten(-2).long()]

    k = nibbles(tiles[..., :half].reshape(n, H, D // 32, B, 16))   # [n, H, D / 32, B, 32]
    k = k.permute(1, 0, 3, 2, 4).reshape(H, n * B, D)
    v = nibbles(tiles[..., half:2 * half].reshape(n, H, D, B // 2)).permute(1, 0, 3, 2)
    v = v.reshape(H, n * B, D)
    sc = tiles[..., 2 * half:].contiguous().view(torch.float8_e4m3fn).float()
    ks = sc[..., :ns].reshape(n, H, B, D // 16).permute(1, 0, 2, 3).reshape(H, n * B, D // 16)
    vs = sc[..., ns:].reshape(n, H, D // 16, B).permute(1, 0, 3, 2).reshape(H, n * B, D // 16)
    k = (k.unflatten(-1, (-1, 16)) * ks.unsqueeze(-1)).flatten(-2) * 2.0 ** k_exp
    v = (v.unflatten(-1, (-1, 16)) * vs.unsqueeze(-1)).flatten(-2) * 2.0 ** v_exp
    return k, v


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _prepare_attention(c, seed):
    g = _gen(seed)
    ctx, win = _attention_layout(c)
    B, D, H = c["block"], c["d"], c["hkv"]
    dt = DTYPES[c["dtype"]]
    need = [-(-t // B) for t in ctx]
    pages = sum(need) + 3
    per = max(max(need), 1)
    page_bytes = B * D + B * D // 8
    pool = torch.empty((pages, H, page_bytes), dtype=torch.uint8, device=DEV)
    # keys and values of unit size and of the size that v_exp stands for
    step = max(1, (1 << 24) // (B * H * D))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        kc, ks = _encode(_randn((m, B, H, D), g).bfloat16().float(), c["k_exp"])
        vc, vs = _encode(_randn((m, B, H, D), g, scale=2.0 ** c["v_exp"]).bfloat16().float(),
                         c["v_exp"])
        pool[p:p + m] = _pack_pages(kc, ks, vc, vs)
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((c["batch"], per), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    start = [0]
    for n in win:
        start.append(start[-1] + n)
    total = start[-1]
    s = dict(case=c, ctx=ctx, win=win, q=_randn((total, c["hq"], D), g, dt),
             k_win=_randn((total, H, D), g, dt),
             v_win=_randn((total, H, D), g, dt, scale=2.0 ** c["v_exp"]), pool=pool, table=table,
             ctx_len=_int32(ctx), q_start=_int32(start), max_q=max(win), max_ctx=max(ctx))
    if own:
        from block_causal_kv_gb300 import d2f
        s["workspace"] = d2f.attn_kv4_workspace(
            torch.device(DEV), batch=c["batch"], total_q=total, max_q_per_seq=s["max_q"],
            max_ctx=s["max_ctx"], num_heads_q=c["hq"], num_heads_kv=H, head_dim=D, block_size=B,
            dtype=d2f.BF16 if dt == torch.bfloat16 else d2f.F32)
    return s


def _prepare_cache(c, seed):
    g = _gen(seed)
    lens = _cache_layout(c)
    B, D, H = c["block"], c["d"], c["hkv"]
    dt = DTYPES[c["dtype"]]
    total = sum(lens)
    pages = sum(-(-n // B) for n in lens)
    free = torch.randperm(pages + 5, generator=g, device=DEV)[:pages]
    src, rows, page_of, off = [], [], [], []
    at = 0
    for n in lens:
        for t in range(0, n, B):
            m = min(B, n - t)
            page_of += [len(src)] * m
            off += list(range(m))
            src.append(at + t)
            rows.append(m)
        at += n
    slot = free[torch.tensor(page_of, device=DEV)] * B + torch.tensor(off, device=DEV)
    return dict(case=c, k=_randn((total, H, D), g, dt, scale=2.0 ** c["k_exp"]),
                v=_randn((total, H, D), g, dt, scale=2.0 ** c["v_exp"]), src_row=_int32(src),
                dst_page=free.int(), n_rows=_int32(rows), slot=slot,
                pool=torch.zeros((pages + 5, H, B * D + B * D // 8), dtype=torch.uint8, device=DEV))


def _prepare_pages(c, seed):
    g = _gen(seed)
    new, cached, free = _pages_layout(c)
    B = c["block"]
    per = max(k + -(-n // B) for n, k in zip(new, cached))
    table = torch.full((c["batch"], max(per, 1)), -1, dtype=torch.int32, device=DEV)
    held = sum(cached)
    order = torch.randperm(held + free + 1, generator=g, device=DEV).int()
    at = 0
    for b, k in enumerate(cached):
        table[b, :k] = order[at:at + k]
        at += k
    return dict(case=c, num_new=_int32(new), ctx_len=_int32([k * B for k in cached]), table=table,
                free_pages=order[held:].contiguous(), free_count=_int32([free]),
                capacity=sum(new) + 3, max_append=sum(-(-n // B) for n in new) + 1)


def _prepare_logprobs(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    R, V = c["rows"], c["vocab"]
    buf = torch.empty((R, V + c["pad"]), dtype=dt, device=DEV)
    for r in range(0, R, 64):
        m = min(64, R - r)
        x = _randn((m, V + c["pad"]), g, scale=3.0)
        peak = torch.randint(0, V, (m, 1), generator=g, device=DEV)
        top = x[:, :V].amax(1, keepdim=True) + 2 + 10 * torch.rand((m, 1), generator=g, device=DEV)
        x.scatter_(1, peak, top)
        buf[r:r + m] = x.to(dt)
    logits = buf[:, :V]
    # committed tokens: the greedy one nine times of ten, else any
    tok = logits.float().argmax(1)
    other = torch.randint(0, V, (R,), generator=g, device=DEV)
    tok = torch.where(torch.rand(R, generator=g, device=DEV) < 0.9, tok, other)
    given = torch.tensor(_given_rows(c), device=DEV)
    tok = torch.where(given, tok, torch.full_like(tok, -1)).int()
    s = dict(case=c, logits=logits, tokens=tok)
    if own:
        from block_causal_kv_gb300 import d2f
        s["workspace"] = d2f.logprobs_workspace(
            torch.device(DEV), n=R, vocab=V, top_k=c["top"],
            dtype=d2f.BF16 if dt == torch.bfloat16 else d2f.F32)
    return s


def prepare(case, seed):
    return {"attention": _prepare_attention, "cache": _prepare_cache, "pages": _prepare_pages,
            "logprobs": _prepare_logprobs}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_attention(s):
    c = s["case"]
    B, D, H, G = c["block"], c["d"], c["hkv"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    r = 0
    for b, (t, n) in enumerate(zip(s["ctx"], s["win"])):
        q = s["q"][r:r + n].float().view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        kw = s["k_win"][r:r + n].float().transpose(0, 1)
        vw = s["v_win"][r:r + n].float().transpose(0, 1)
        if t:
            tiles = s["pool"][s["table"][b, :-(-t // B)].long()]
            k, v = _decode_pages(tiles, B, D, c["k_exp"], c["v_exp"])
            k, v = torch.cat([k[:, :t], kw], 1), torch.cat([v[:, :t], vw], 1)
        else:
            k, v = kw, vw
        x = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        blk = torch.arange(n, device=DEV) // B
        hide = (blk[None, :] > blk[:, None]).repeat_interleave(G, 0)
        x[:, :, t:].masked_fill_(hide, float("-inf"))
        m = x.amax(-1, keepdim=True)
        p = (x - m).exp_()
        l = p.sum(-1, keepdim=True)
        o = (p @ v) / l
        out[r:r + n] = o.view(H, n, G, D).permute(1, 0, 2, 3).reshape(n, H * G, D).to(out.dtype)
        lse[r:r + n] = (m + l.log()).view(H, n, G).permute(1, 0, 2).reshape(n, H * G)
        r += n
    return out, lse


def _plain_cache(s):
    c = s["case"]
    B, D = c["block"], c["d"]
    rows = s["src_row"].long()[:, None] + torch.arange(B, device=DEV)
    live = torch.arange(B, device=DEV) < s["n_rows"].long()[:, None]
    rows = torch.where(live, rows, torch.zeros_like(rows))
    codes = []
    for x, e in ((s["k"], c["k_exp"]), (s["v"], c["v_exp"])):
        blocks = torch.where(live[:, :, None, None], x[rows].float(), 0.0)
        codes += list(_encode(blocks, e))
    s["pool"][s["dst_page"].long()] = _pack_pages(*codes)
    page, off = s["slot"] // B, s["slot"] % B
    used, at = torch.unique(page, return_inverse=True)
    k, v = _decode_pages(s["pool"][used], B, D, c["k_exp"], c["v_exp"])
    at = at * B + off
    dt = s["k"].dtype
    return k[:, at].transpose(0, 1).to(dt), v[:, at].transpose(0, 1).to(dt)


def _plain_pages(s):
    c = s["case"]
    B = c["block"]
    new, ctx = s["num_new"].long(), s["ctx_len"].long()
    need = (new + B - 1) // B
    fits = ctx // B + need <= s["table"].shape[1]
    need = torch.where(fits, need, torch.zeros_like(need))
    end = need.cumsum(0)
    ok = fits & (end <= s["free_count"].long())
    need = torch.where(ok, need, torch.zeros_like(need))
    first = need.cumsum(0) - need
    row_start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), new.cumsum(0)])
    n = int(need.sum())
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), need)
    i = torch.arange(n, device=DEV) - first[req]
    page = s["free_pages"][s["free_count"].long() - 1 - torch.arange(n, device=DEV)]
    table = s["table"].clone()
    table[req, ctx[req] // B + i] = page
    app = torch.full((3, s["max_append"]), -1, dtype=torch.int32, device=DEV)
    app[0, :n] = (row_start[req] + i * B).int()
    app[1, :n] = page
    app[2] = 0
    app[2, :n] = torch.minimum(new[req] - i * B, torch.full_like(i, B)).int()
    slot = torch.full((s["capacity"],), -1, dtype=torch.long, device=DEV)
    total = int(row_start[-1])
    tok_req = torch.repeat_interleave(torch.arange(len(new), device=DEV), new)
    t = torch.arange(total, device=DEV) - row_start[tok_req]
    live = ok[tok_req]
    at = table[tok_req[live], ctx[tok_req[live]] // B + t[live] // B].long()
    slot[:total][live] = at * B + t[live] % B
    return dict(page_table=table, ctx_len=(ctx + torch.where(ok, new, 0)).int(),
                row_start=row_start.int(), admitted=ok.byte(), slot=slot, app_src=app[0],
                app_dst=app[1], app_rows=app[2], n_append=_int32([n]),
                free_count=(s["free_count"] - n).int())


def _plain_logprobs(s):
    c = s["case"]
    R, k = c["rows"], c["top"]
    lp = torch.zeros(R, dtype=torch.float32, device=DEV)
    ent = torch.zeros(R, dtype=torch.float32, device=DEV)
    ids = torch.full((R, k), -1, dtype=torch.int32, device=DEV)
    tlp = torch.zeros((R, k), dtype=torch.float32, device=DEV)
    at = (s["tokens"] >= 0).nonzero()[:, 0]
    x = s["logits"][at].float()
    x = x - x.amax(1, keepdim=True)
    e = x.exp()
    total = e.sum(1)
    ln = total.log()
    lp[at] = x.gather(1, s["tokens"][at].long()[:, None])[:, 0] - ln
    ent[at] = ln - (e * x).sum(1) / total
    if k:
        v, i = x.sort(dim=1, descending=True, stable=True)
        ids[at] = i[:, :k].int()
        tlp[at] = v[:, :k] - ln[:, None]
    return dict(logprob=lp, entropy=ent, top_id=ids, top_logprob=tlp)


def _own(s):
    from block_causal_kv_gb300 import d2f
    c = s["case"]
    if c["op"] == "attention":
        return d2f.block_attn_kv4(s["q"], s["k_win"], s["v_win"], s["pool"], s["table"],
                                  s["ctx_len"], s["q_start"], block_size=c["block"],
                                  max_q_per_seq=s["max_q"], max_ctx=s["max_ctx"],
                                  k_exp=c["k_exp"], v_exp=c["v_exp"], workspace=s["workspace"])
    if c["op"] == "cache":
        d2f.kv4_append(s["k"], s["v"], s["src_row"], s["dst_page"], s["pool"],
                       block_size=c["block"], n_rows=s["n_rows"], k_exp=c["k_exp"],
                       v_exp=c["v_exp"])
        return d2f.kv4_read(s["pool"], s["slot"], head_dim=c["d"], block_size=c["block"],
                            dtype=s["k"].dtype, k_exp=c["k_exp"], v_exp=c["v_exp"])
    if c["op"] == "pages":
        return d2f.page_map(s["num_new"], s["ctx_len"], s["table"], s["free_pages"],
                            s["free_count"], block_size=c["block"], capacity=s["capacity"],
                            max_append=s["max_append"])
    return d2f.token_logprobs(s["logits"], s["tokens"], top_k=c["top"],
                              workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "cache": _plain_cache, "pages": _plain_pages,
            "logprobs": _plain_logprobs}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_table():
    vals = []
    for bits in range(256):
        e, m = (bits >> 3) & 15, bits & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        vals.append(float("nan") if bits & 127 == 127 else -x if bits & 128 else x)
    return torch.tensor(vals, dtype=torch.float64, device=DEV)


def _exact_tokens(pool, page, off, h, B, D, k_exp, v_exp):
    """K and V float64 [n, D] of head h at (page, offset in it), byte by byte."""
    value = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    scale = _e4m3_table()
    tile = pool[page, h].long()
    d = torch.arange(D, device=DEV)[None, :]
    o = off[:, None]
    kb = tile.gather(1, (d // 32) * (B * 16) + o * 16 + (d % 32) // 2)
    vb = tile.gather(1, B * D // 2 + d * (B // 2) + o // 2)
    ks = tile.gather(1, B * D + o * (D // 16) + d // 16)
    vs = tile.gather(1, B * D + B * D // 16 + (d // 16) * B + o)
    k = value[torch.where(d % 2 == 0, kb % 16, kb // 16)] * scale[ks] * 2.0 ** k_exp
    v = value[torch.where(o % 2 == 0, vb % 16, vb // 16)] * scale[vs] * 2.0 ** v_exp
    return k, v


def _exact_attention(c, seed):
    s = _prepare_attention(c, seed)
    B, D, G = c["block"], c["d"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    r = 0
    for b, (t, n) in enumerate(zip(s["ctx"], s["win"])):
        tok = torch.arange(t, device=DEV)
        page = s["table"][b].long()[tok // B]
        blk = torch.arange(n, device=DEV) // B
        see = torch.cat([torch.ones((n, t), dtype=torch.bool, device=DEV),
                         blk[None, :] <= blk[:, None]], 1)
        for h in range(c["hkv"]):
            kc, vc = _exact_tokens(s["pool"], page, tok % B, h, B, D, c["k_exp"], c["v_exp"])
            k = torch.cat([kc, s["k_win"][r:r + n, h].double()])
            v = torch.cat([vc, s["v_win"][r:r + n, h].double()])
            q = s["q"][r:r + n, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,kd->ngk", q, k) / math.sqrt(D)
            x = torch.where(see[:, None, :], x, float("-inf"))
            z = torch.logsumexp(x, -1)
            lse[r:r + n, h * G:(h + 1) * G] = z
            out[r:r + n, h * G:(h + 1) * G] = torch.einsum("ngk,kd->ngd",
                                                           (x - z[..., None]).exp(), v)
        r += n
    return out, lse


def _exact_cache(c, seed):
    s = _prepare_cache(c, seed)
    grid = torch.tensor(_E2M1[:8], dtype=torch.float64, device=DEV)
    mids = (grid[1:] + grid[:-1]) / 2
    e4m3 = _e4m3_table()[:127]
    e_mid = (e4m3[1:] + e4m3[:-1]) / 2

    def nearest(x, levels, mid):
        """Index of the level nearest to x >= 0, ties to the even index."""
        lo, hi = torch.bucketize(x, mid), torch.bucketize(x, mid, right=True)
        return torch.where(lo % 2 == 0, lo, hi)

    def quantised(x, exp):
        outs = []
        for part in x.split(2048):
            y = part.double().unflatten(-1, (-1, 16)) / 2.0 ** exp
            sc = e4m3[nearest(y.abs().amax(-1, keepdim=True) / 6, e4m3, e_mid)]
            z = torch.where(sc > 0, y.abs() / torch.where(sc > 0, sc, 1.0), 0.0)
            val = grid[nearest(z, grid, mids)] * sc * torch.sign(y) * 2.0 ** exp
            outs.append(val.flatten(-2))
        return torch.cat(outs)

    return quantised(s["k"], c["k_exp"]), quantised(s["v"], c["v_exp"])


def exact(case, seed):
    c = case
    if c["op"] == "attention":
        return _exact_attention(c, seed)
    if c["op"] == "cache":
        return _exact_cache(c, seed)
    if c["op"] == "pages":
        return None
    s = _prepare_logprobs(c, seed)
    R, k = c["rows"], c["top"]
    out = dict(logprob=torch.zeros(R, dtype=torch.float64, device=DEV),
               entropy=torch.zeros(R, dtype=torch.float64, device=DEV),
               top_id=torch.full((R, k), -1, dtype=torch.int32, device=DEV),
               top_logprob=torch.zeros((R, k), dtype=torch.float64, device=DEV))
    for r in range(R):
        t = int(s["tokens"][r])
        if t < 0:
            continue
        lp = s["logits"][r].double()
        lp = lp - torch.logsumexp(lp, 0)
        out["logprob"][r] = lp[t]
        out["entropy"][r] = -(lp.exp() * lp).sum()
        if k:
            ids = torch.argsort(-lp, stable=True)[:k]
            out["top_id"][r] = ids.int()
            out["top_logprob"][r] = lp[ids]
    return out

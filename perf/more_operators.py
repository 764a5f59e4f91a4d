"""Cases that measure the attention of prompts (packed requests, optionally behind a cached
prefix), the attention of one new token a sequence over the paged cache, and the store of token
rows into that cache.

Shapes are those of this repository's workloads (LLaDA-8B-shaped layers: 32 heads, head_dim 128;
Dream-7B-shaped: 28 query heads on 4 KV heads; pages of 8, 16 or 32 tokens; contexts up to 32,768)
or generic. `run` computes an operator in plain torch operations while `own` is false and calls
block_causal_kv_gb300.d2f while it is true.

The cache is [pages][KV heads][page size][head_dim] for K and for V; token t of sequence b is row
t % page size of page table[b][t / page size].
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG_INF = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# prompts: `new` rows a request (from new_min on), behind `ctx` cached tokens (from ctx_min on);
# row i sees the cached tokens and the new rows j with j // see <= i // see (1: causal, 0: all)
def listed():
    return [
        # the smallest layer of this repository's workloads, float32: one short prompt
        dict(name="prompt_tiny", op="prompt", dtype="f32", batch=1, hq=4, hkv=4, d=64, block=16,
             new=100, new_min=100, ctx=0, ctx_min=0, see=1, layout=1),
        # one request's prompt, blocks of 16 seen in both directions, earlier ones by later ones
        dict(name="prompt_llada", op="prompt", dtype="bf16", batch=1, hq=32, hkv=32, d=128,
             block=16, new=1024, new_min=1024, ctx=0, ctx_min=0, see=16, layout=2),
        # the prompts of a served batch, of every length, causal, grouped heads
        dict(name="prompt_ragged", op="prompt", dtype="bf16", batch=16, hq=32, hkv=8, d=128,
             block=16, new=4096, new_min=251, ctx=0, ctx_min=0, see=1, layout=3),
        # one long document, causal: the products bound it
        dict(name="prompt_long", op="prompt", dtype="bf16", batch=1, hq=28, hkv=4, d=128, block=16,
             new=16384, new_min=16384, ctx=0, ctx_min=0, see=1, layout=4),
        # a few new rows of two requests behind long cached prefixes (a chat's next turn)
        dict(name="prompt_prefix", op="prompt", dtype="bf16", batch=2, hq=28, hkv=4, d=128,
             block=16, new=77, new_min=40, ctx=32768, ctx_min=20000, see=1, layout=5),
        # one token of one short request, float32
        dict(name="token_tiny", op="token", dtype="f32", batch=1, hq=4, hkv=4, d=64, block=16,
             ctx=64, ctx_min=64, layout=6),
        # one token of one request: latency of a single layer
        dict(name="token_llada", op="token", dtype="bf16", batch=1, hq=32, hkv=32, d=128, block=16,
             ctx=1024, ctx_min=1024, layout=7),
        # a served batch with contexts of every length, partly filled last pages
        dict(name="token_ragged", op="token", dtype="bf16", batch=16, hq=32, hkv=32, d=128,
             block=16, ctx=4096, ctx_min=251, layout=8),
        # grouped heads, a larger batch of equal contexts
        dict(name="token_dream", op="token", dtype="bf16", batch=64, hq=28, hkv=4, d=128, block=32,
             ctx=8192, ctx_min=8192, layout=9),
        # the longest contexts: the cache read bounds it
        dict(name="token_long", op="token", dtype="bf16", batch=4, hq=32, hkv=32, d=128, block=16,
             ctx=32768, ctx_min=32768, layout=10),
        # one decode step's new tokens, one a request
        dict(name="store_step", op="store", dtype="bf16", batch=8, hkv=4, d=128, block=16,
             tokens=1, tokens_min=1, layout=11),
        # the prompts of a served batch, of every length
        dict(name="store_prompts", op="store", dtype="bf16", batch=16, hkv=32, d=128, block=16,
             tokens=4096, tokens_min=251, layout=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


_HEADS = [(32, 32), (28, 4), (4, 4), (8, 2), (32, 8), (5, 1)]


def _draw_prompt(rng):
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hkv = rng.choice(_HEADS)
    new = _log_int(rng, 1, 16384 if dtype == "bf16" else 1024)
    ctx = _log_int(rng, 1, 32768 if dtype == "bf16" else 1024) if rng.random() < 0.4 else 0
    return dict(op="prompt", dtype=dtype, batch=_log_int(rng, 1, 16), hq=hq, hkv=hkv,
                d=rng.choice([64, 128, 128]), block=rng.choice([8, 16, 16, 32]), new=new,
                new_min=rng.choice([new, rng.randint(1, new)]), ctx=ctx,
                ctx_min=rng.choice([ctx, rng.randint(0, ctx)]),
                see=rng.choice([0, 1, 1, 1, 8, 16, 32, rng.randint(2, 100)]),
                layout=rng.randrange(1 << 30))


def _draw_token(rng):
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hkv = rng.choice(_HEADS)
    ctx = _log_int(rng, 1, 32768 if dtype == "bf16" else 4096)
    return dict(op="token", dtype=dtype, batch=_log_int(rng, 1, 64), hq=hq, hkv=hkv,
                d=rng.choice([64, 128, 128]), block=rng.choice([8, 16, 16, 32]), ctx=ctx,
                ctx_min=rng.choice([ctx, rng.randint(0, ctx)]), layout=rng.randrange(1 << 30))


def _draw_store(rng):
    tokens = _log_int(rng, 1, 4096)
    return dict(op="store", dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_log_int(rng, 1, 16),
                hkv=rng.choice([1, 2, 4, 8, 32]), d=rng.choice([64, 128]),
                block=rng.choice([8, 16, 32]), tokens=tokens, tokens_min=rng.randint(1, tokens),
                layout=rng.randrange(1 << 30))


def draw(rng):
    make = rng.choice([_draw_prompt, _draw_prompt, _draw_token, _draw_token, _draw_store])
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


def _lengths(c):
    """New rows and cached tokens of each request."""
    rng = random.Random(c["layout"])
    if c["op"] == "store":
        return _spread(rng, c["batch"], c["tokens_min"], c["tokens"]), [0] * c["batch"]
    ctx = _spread(rng, c["batch"], c["ctx_min"], c["ctx"])
    if c["op"] == "token":
        return [1] * c["batch"], ctx
    return _spread(rng, c["batch"], c["new_min"], c["new"]), ctx


def _seen(n, t, see):
    """Pairs (row, key) of one request."""
    if see == 0:
        return n * (n + t)
    whole, rest = divmod(n, see)
    return n * t + see * see * whole * (whole + 1) // 2 + rest * n


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    new, ctx = _lengths(c)
    rows, toks = sum(new), sum(ctx)
    kv = 2 * c["hkv"] * c["d"] * e
    if c["op"] == "store":
        return {"bytes": 2 * rows * kv + 8 * rows, "flops": 0}
    pages = sum(-(-t // c["block"]) for t in ctx)
    data = 2 * rows * c["hq"] * c["d"] * e + 4 * rows * c["hq"] + (rows + toks) * kv
    ints = 4 * (pages + 2 * c["batch"] + 1)
    if c["op"] == "token":   # the new token's K and V go to its page
        return {"bytes": data + ints + rows * kv, "flops": 4 * c["d"] * c["hq"] * (toks + rows)}
    seen = sum(_seen(n, t, c["see"]) for n, t in zip(new, ctx))
    return {"bytes": data + ints, "flops": 4 * c["d"] * c["hq"] * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _fill(shape, g, dtype):
    """Unit-size values, made a slice at a time."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    step = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        out[i:i + step] = _randn((min(step, shape[0] - i),) + tuple(shape[1:]), g, dtype)
    return out


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(c, lens, g):
    """A pool of shuffled pages, the page table of `lens` tokens a sequence."""
    need = [-(-t // c["block"]) for t in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((c["batch"], max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return (pages, c["hkv"], c["block"], c["d"]), table


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    new, ctx = _lengths(c)
    rows = sum(new)
    s = dict(case=c, new=new, ctx=ctx, k=_randn((rows, c["hkv"], c["d"]), g, dt),
             v=_randn((rows, c["hkv"], c["d"]), g, dt))
    if c["op"] == "store":
        shape, table = _pages(c, new, g)
        at = [torch.arange(n, device=DEV) for n in new]
        s["slot"] = torch.cat([table[b].long()[t // c["block"]] * c["block"] + t % c["block"]
                               for b, t in enumerate(at)])
        s["k_pool"] = torch.zeros(shape, dtype=dt, device=DEV)
        s["v_pool"] = torch.zeros(shape, dtype=dt, device=DEV)
        return s
    # queries a little larger than unit size: some keys stand out of their row's softmax
    s["q"] = (_randn((rows, c["hq"], c["d"]), g, torch.float32) * 1.5).to(dt)
    shape, table = _pages(c, [t + 1 for t in ctx] if c["op"] == "token" else ctx, g)
    s["k_pool"], s["v_pool"], s["table"] = _fill(shape, g, dt), _fill(shape, g, dt), table
    s["ctx_len"] = _int32(ctx)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["row_start"] = _int32(start)
    if own:
        from block_causal_kv_gb300 import d2f
        kw = dict(batch=c["batch"], max_ctx=max(ctx), num_heads_q=c["hq"], num_heads_kv=c["hkv"],
                  head_dim=c["d"], block_size=c["block"],
                  dtype=d2f.BF16 if dt == torch.bfloat16 else d2f.F32)
        if c["op"] == "prompt":
            s["workspace"] = d2f.prompt_attn_workspace(torch.device(DEV), rows=rows, **kw)
        else:
            s["workspace"] = d2f.token_attn_workspace(torch.device(DEV), **kw)
    return s


# ---------------------------------------------------------------------------
# one pass, plain
# ---------------------------------------------------------------------------
def _cached(s, b):
    """K and V float32 [Hkv, tokens, D] of sequence b's cached tokens."""
    t, B = s["ctx"][b], s["case"]["block"]
    at = s["table"][b, :-(-t // B)].long()
    return tuple(p[at].transpose(0, 1).flatten(1, 2)[:, :t].float() for p in (s["k_pool"],
                                                                              s["v_pool"]))


def _plain_attention(s, see):
    c = s["case"]
    D, H, G = c["d"], c["hkv"], c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    r = 0
    for b, (n, t) in enumerate(zip(s["new"], s["ctx"])):
        kc, vc = _cached(s, b)
        k = torch.cat([kc, s["k"][r:r + n].float().transpose(0, 1)], 1)
        v = torch.cat([vc, s["v"][r:r + n].float().transpose(0, 1)], 1)
        step = max(1, (1 << 28) // (c["hq"] * (n + t)))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            m = i1 - i0
            last = n if see == 0 else min(n, ((i1 - 1) // see + 1) * see)
            q = s["q"][r + i0:r + i1].float().view(m, H, G, D).permute(1, 2, 0, 3)
            x = (q.reshape(H, G * m, D) @ k[:, :t + last].transpose(1, 2)) * (1.0 / math.sqrt(D))
            if see:
                i = torch.arange(i0, i1, device=DEV) // see
                j = torch.arange(last, device=DEV) // see
                x[:, :, t:].masked_fill_((j[None, :] > i[:, None]).repeat(G, 1), NEG_INF)
            top = x.amax(-1, keepdim=True)
            p = x.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = (p @ v[:, :t + last]) / total
            o = o.view(H, G, m, D).permute(2, 0, 1, 3).reshape(m, H * G, D)
            z = (top + total.log()).view(H, G, m).permute(2, 0, 1).reshape(m, H * G)
            out[r + i0:r + i1] = o.to(out.dtype)
            lse[r + i0:r + i1] = z
        r += n
    return out, lse


def _plain_token(s):
    out, lse = _plain_attention(s, 0)
    B = s["case"]["block"]
    t = s["ctx_len"].long()
    page = s["table"].gather(1, (t // B)[:, None])[:, 0].long()
    s["k_pool"][page, :, t % B] = s["k"]
    s["v_pool"][page, :, t % B] = s["v"]
    return out, lse, s["k_pool"], s["v_pool"]


def _plain_store(s):
    B = s["case"]["block"]
    page, off = s["slot"] // B, s["slot"] % B
    s["k_pool"][page, :, off] = s["k"]
    s["v_pool"][page, :, off] = s["v"]
    return s["k_pool"], s["v_pool"]


# ---------------------------------------------------------------------------
# one pass, the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    from block_causal_kv_gb300 import d2f
    c = s["case"]
    if c["op"] == "store":
        d2f.kv_store(s["k"], s["v"], s["slot"], s["k_pool"], s["v_pool"], block_size=c["block"])
        return s["k_pool"], s["v_pool"]
    if c["op"] == "token":
        out, lse = d2f.token_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx_len"],
                                  k_new=s["k"], v_new=s["v"], block_size=c["block"],
                                  max_ctx=max(s["ctx"]), workspace=s["workspace"])
        return out, lse, s["k_pool"], s["v_pool"]
    if c["ctx"] == 0:
        return d2f.prompt_attn(s["q"], s["k"], s["v"], s["row_start"], mask_block=c["see"],
                               workspace=s["workspace"])
    return d2f.prompt_attn(s["q"], s["k"], s["v"], s["row_start"], mask_block=c["see"],
                           k_pool=s["k_pool"], v_pool=s["v_pool"], page_table=s["table"],
                           ctx_len=s["ctx_len"], block_size=c["block"], max_ctx=max(s["ctx"]),
                           workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "store":
        return _plain_store(state)
    if op == "token":
        return _plain_token(state)
    return _plain_attention(state, state["case"]["see"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_heads(s, see):
    """Head by head, token by token through the page table."""
    c = s["case"]
    B, D, G = c["block"], c["d"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    r = 0
    for b, (n, t) in enumerate(zip(s["new"], s["ctx"])):
        tok = torch.arange(t, device=DEV)
        page, off = s["table"][b].long()[tok // B], tok % B
        for h in range(c["hkv"]):
            k = torch.cat([s["k_pool"][page, h, off], s["k"][r:r + n, h]]).double()
            v = torch.cat([s["v_pool"][page, h, off], s["v"][r:r + n, h]]).double()
            for i0 in range(0, n, 512):
                i = torch.arange(i0, min(n, i0 + 512), device=DEV)
                end = n if see == 0 else min(n, (int(i[-1]) // see + 1) * see)
                j = torch.arange(end, device=DEV)
                sight = torch.ones((len(i), t + end), dtype=torch.bool, device=DEV)
                if see:
                    sight[:, t:] = (i[:, None] // see) >= (j[None, :] // see)
                q = s["q"][r + i, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,kd->igk", q, k[:t + end]) / math.sqrt(D)
                x = torch.where(sight[:, None, :], x, NEG_INF)
                z = torch.logsumexp(x, -1)
                lse[r + i, h * G:(h + 1) * G] = z
                out[r + i, h * G:(h + 1) * G] = torch.einsum(
                    "igk,kd->igd", torch.exp(x - z[..., None]), v[:t + end])
        r += n
    return out, lse


def exact(case, seed):
    c = case
    if work(c)["flops"] > 3e12:   # over a few seconds in 64 bits
        return None
    s = prepare(c, seed)
    B = c["block"]
    if c["op"] == "prompt":
        return _exact_heads(s, c["see"])
    # the pools: copies, exact in their own type
    if c["op"] == "token":
        out, lse = _exact_heads(s, 0)
        slot = [int(s["table"][b, t // B]) * B + t % B for b, t in enumerate(s["ctx"])]
    else:
        slot = s["slot"].tolist()
    at = torch.tensor(slot, device=DEV)
    pools = []
    for pool, x in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
        flat = pool.transpose(1, 2).reshape(-1, c["hkv"], c["d"]).clone()
        flat[at] = x
        pools.append(flat.view(-1, B, c["hkv"], c["d"]).transpose(1, 2).contiguous())
    return (out, lse, *pools) if c["op"] == "token" else tuple(pools)

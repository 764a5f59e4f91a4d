"""d2f_kv_store: bitwise copies into slots, bounds of indices, and prompts that the page map laid
out running into D2F windows and into single-token steps."""
import pytest
import torch

from gpu_common import check_attention, device

import oracle
from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,hkv,D,B", [
    (1, 1, 128, 16), (8, 4, 128, 16), (1000, 32, 128, 16), (77, 3, 64, 8), (50, 2, 32, 1),
    (33, 5, 80, 7), (9, 1, 5, 3), (40, 2, 129, 256), (0, 2, 64, 16)])
def test_rows_go_to_their_slots(n, hkv, D, B, dtype):
    dev = device()
    g = torch.Generator().manual_seed(n + D)
    pages = n // B + 4
    k, v = (torch.randn((n, hkv, D), generator=g).to(dtype) for _ in range(2))
    kp, vp = (torch.randn((pages, hkv, B, D), generator=g).to(dtype) for _ in range(2))
    slot = torch.randperm(pages * B, generator=g)[:n]
    slot[::3] = -1
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    gk, gv = kp.to(dev), vp.to(dev)
    d2f.kv_store(k.to(dev), v.to(dev), slot.to(dev), gk, gv, block_size=B, err=err)
    torch.cuda.synchronize()
    at = (slot >= 0).nonzero()[:, 0]
    kp[slot[at] // B, :, slot[at] % B], vp[slot[at] // B, :, slot[at] % B] = k[at], v[at]
    assert torch.equal(gk.cpu(), kp) and torch.equal(gv.cpu(), vp) and int(err) == 0


@pytest.mark.parametrize("bad", [-2, 64, 10 ** 12, -2 ** 62])
def test_slots_outside_the_pool(bad):
    dev = device()
    k = torch.randn((3, 2, 64), device=dev).bfloat16()
    pad = torch.full((8, 2, 16, 64), 7.0, device=dev).bfloat16()
    kp, vp = pad[2:6].clone(), pad[2:6].clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    d2f.kv_store(k, k, torch.tensor([5, bad, 63], device=dev), kp, vp, block_size=16, err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    want = pad[2:6].clone()
    want[0, :, 5], want[3, :, 15] = k[0], k[2]
    assert torch.equal(kp, want) and torch.equal(vp, want)


def test_pools_past_32_bits():
    """Slots whose elements lie past 2^31 and 2^32 of the pool."""
    dev = device()
    pages, B, D = 1 << 17, 256, 128                      # 2^32 elements
    kp = torch.zeros((pages + 3, 1, B, D), dtype=BF, device=dev)
    k = torch.randn((4, 1, D), device=dev).bfloat16()
    slot = torch.tensor([0, (1 << 24) + 5, (pages + 2) * B + 255, (1 << 25) + 77], device=dev)
    d2f.kv_store(k, k, slot, kp, kp, block_size=B)
    flat = kp.view(-1, D)
    assert torch.equal(flat[slot], k[:, 0])
    assert int((flat != 0).any(1).sum()) == 4


@pytest.mark.parametrize("dtype", [BF, F32])
def test_refusals(dtype):
    dev = device()
    k = torch.zeros((3, 2, 64), dtype=dtype, device=dev)
    kp = torch.zeros((4, 2, 16, 64), dtype=dtype, device=dev)
    slot = torch.zeros(3, dtype=torch.int64, device=dev)
    for args in ((k[:2], k, slot, kp, kp), (k, k, slot.int(), kp, kp), (k, k, slot[:2], kp, kp),
                 (k, k, slot, kp[:, :1], kp), (k, k.half(), slot, kp, kp), (k, k, slot.cpu(), kp, kp)):
        with pytest.raises((ValueError, TypeError)):
            d2f.kv_store(*args, block_size=16)
    with pytest.raises(ValueError):
        d2f.kv_store(k, k, slot, kp, kp, block_size=8)


def dense(q, k, v, see):
    """float64 attention of rows over keys, see [rows, keys] bool."""
    G = q.shape[1] // k.shape[1]
    k, v = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    x = torch.einsum("rhd,khd->hrk", q.double(), k) * q.shape[2] ** -0.5
    x = x.masked_fill(~see, float("-inf"))
    return (torch.einsum("hrk,khd->rhd", x.softmax(-1), v), x.logsumexp(-1).T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 128), (3, 3, 64)])
def test_prompts_then_windows_and_tokens(hq, hkv, D, dtype):
    """Two turns of two requests: the page map lays the prompts out, their attention runs, their rows
    are stored; a D2F window and then single tokens read the same cache; a second prompt comes
    behind the first's cached blocks. All against attention over the plain rows."""
    dev = device()
    B, lens = 16, [48, 80]
    g = torch.Generator().manual_seed(D)

    def draw(*shape):
        return torch.randn(shape, generator=g).to(dtype)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)
    pages = 24
    kp, vp = draw(pages, hkv, B, D).to(dev), draw(pages, hkv, B, D).to(dev)
    table = torch.full((2, 12), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=g).int().to(dev)
    count = i32([pages])
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ctx = i32([0, 0])
    keys = [torch.zeros((0, hkv, D), dtype=dtype)] * 2
    vals = list(keys)
    for turn, new in enumerate((lens, [21, 5])):
        rows = sum(new)
        m = d2f.page_map(i32(new), ctx, table, free, count, block_size=B, capacity=rows + 4,
                         max_append=12, free_count_out=count, err=err)
        q, k, v = draw(rows + 4, hq, D), draw(rows + 4, hkv, D), draw(rows + 4, hkv, D)
        prefix = {} if turn == 0 else dict(k_pool=kp, v_pool=vp, page_table=table, ctx_len=ctx,
                                           max_ctx=80)
        out, lse = d2f.prompt_attn(q.to(dev), k.to(dev), v.to(dev), m["row_start"], mask_block=B,
                                   block_size=B, err=err, **prefix)
        d2f.kv_store(k.to(dev), v.to(dev), m["slot"], kp, vp, block_size=B, err=err)
        torch.cuda.synchronize()
        r = 0
        for b, n in enumerate(new):
            old = len(keys[b])
            keys[b], vals[b] = torch.cat([keys[b], k[r:r + n]]), torch.cat([vals[b], v[r:r + n]])
            i, j = torch.arange(n) // B, torch.arange(n) // B
            see = torch.cat([torch.ones((n, old), dtype=torch.bool), j[None] <= i[:, None]], 1)
            check_attention(out[r:r + n], lse[r:r + n], *dense(q[r:r + n], keys[b], vals[b], see), dtype)
            r += n
        ctx = m["ctx_len"]
        if turn == 0:   # a window of one block a request reads what was stored
            q, k, v = draw(2 * B, hq, D), draw(2 * B, hkv, D), draw(2 * B, hkv, D)
            out, lse = d2f.block_attn(q.to(dev), k.to(dev), v.to(dev), kp, vp, table, ctx,
                                      i32([0, B, 2 * B]), block_size=B, max_q_per_seq=B, max_ctx=80,
                                      err=err)
            ref, ref_lse = oracle.block_attn(q, k, v, kp.cpu(), vp.cpu(), table.cpu().clamp(min=0),
                                             ctx.cpu(), torch.tensor([0, B, 2 * B], dtype=torch.int32), B)
            check_attention(out, lse, ref, ref_lse, dtype)
            for b in range(2):
                see = torch.ones((B, len(keys[b]) + B), dtype=torch.bool)
                want = dense(q[b * B:b * B + B], torch.cat([keys[b], k[b * B:b * B + B]]),
                             torch.cat([vals[b], v[b * B:b * B + B]]), see)
                check_attention(out[b * B:b * B + B], lse[b * B:b * B + B], *want, dtype)
    for _ in range(9):  # nine tokens: they fill a page and go on in the next
        q, k, v = draw(2, hq, D), draw(2, hkv, D), draw(2, hkv, D)
        for b in range(2):   # the scheduler's part: a page for a token that begins one
            c = int(ctx[b])
            if c % B == 0:
                n = int(count)
                table[b, c // B] = free[n - 1]
                count -= 1
        out, lse = d2f.token_attn(q.to(dev), kp, vp, table, ctx, k_new=k.to(dev), v_new=v.to(dev),
                                  block_size=B, max_ctx=192, err=err)
        ctx = ctx + 1
        torch.cuda.synchronize()
        for b in range(2):
            keys[b], vals[b] = torch.cat([keys[b], k[b:b + 1]]), torch.cat([vals[b], v[b:b + 1]])
            see = torch.ones((1, len(keys[b])), dtype=torch.bool)
            check_attention(out[b:b + 1], lse[b:b + 1], *dense(q[b:b + 1], keys[b], vals[b], see), dtype)
    assert int(err) == 0 and ctx.tolist() == [len(x) for x in keys]

"""d2f_kv4_append and d2f_kv4_read against the format's definition: bytes and values."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def expected_pool(k, v, entries, pages, B, D, k_exp, v_exp):
    hkv = k.shape[1]
    pool = np.zeros((pages, hkv, B * D * 9 // 8), np.uint8)
    for src, dst, m in entries:
        for h in range(hkv):
            kb, vb = np.zeros((B, D)), np.zeros((B, D))
            kb[:m], vb[:m] = k[src:src + m, h].double().numpy(), v[src:src + m, h].double().numpy()
            kc, ks, _ = ref.encode(kb, k_exp)
            vc, vs, _ = ref.encode(vb, v_exp)
            pool[dst, h] = ref.page_tile(kc, ks, vc, vs)
    return pool


def draw(g, rows, hkv, D, dtype):
    """Values of many sizes, with zeros, exact ties of the code grid and tiny groups."""
    x = torch.randn((rows, hkv, D), generator=g)
    x = x * torch.exp2(torch.randint(-12, 8, (rows, hkv, D // 16, 1), generator=g).float()
                       ).expand(-1, -1, -1, 16).reshape(rows, hkv, D)
    grid = torch.tensor([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -2.5, -5.0, 0.5,
                         -6.0, 1e-30, -0.0])
    x[0, 0, :16] = grid
    x[0, 0, 16:32] = 0.0
    for i in range(8):  # ties at every mantissa of the scale: (8 + i) / 8 times the grid
        x[1, 0, 16 * (i % (D // 16)):16 * (i % (D // 16)) + 16] = grid * (8 + i) / 8
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_append_bytes_and_read_back(B, D, hkv, dtype):
    dev = device()
    g = torch.Generator().manual_seed(B * D + hkv)
    rows = 5 * B + 3
    k, v = draw(g, rows, hkv, D, dtype), draw(g, rows, hkv, D, dtype)
    # odd starts, short entries, an empty one, the last rows
    entries = [(0, 4, B), (B + 1, 0, B - 1), (3, 6, 1), (2 * B, 2, 0), (rows - B, 5, B)]
    pages, k_exp, v_exp = 8, 1, -2
    pool = torch.full((pages, hkv, B * D * 9 // 8), 0xA5, dtype=torch.uint8, device=dev)
    err = i32([0], dev)
    d2f.kv4_append(k.to(dev), v.to(dev), i32([e[0] for e in entries], dev),
                   i32([e[1] for e in entries], dev), pool, block_size=B,
                   n_rows=i32([e[2] for e in entries], dev), k_exp=k_exp, v_exp=v_exp, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    got, want = pool.cpu().numpy(), expected_pool(k, v, entries, pages, B, D, k_exp, v_exp)
    written = [e[1] for e in entries]
    for pg in range(pages):
        if pg not in written:
            assert (got[pg] == 0xA5).all()
            continue
        assert np.array_equal(got[pg, :, B * D:], want[pg, :, B * D:]), "scales of page %d" % pg
        assert np.array_equal(got[pg], want[pg]), "codes of page %d" % pg
    # read every slot of the written pages, out of order, with gaps
    slots = [pg * B + o for pg in written for o in range(B)]
    slots = [slots[i] for i in torch.randperm(len(slots), generator=g)] + [-1, slots[0], -1]
    kr, vr = d2f.kv4_read(pool, torch.tensor(slots, device=dev), head_dim=D, block_size=B,
                          dtype=dtype, k_exp=k_exp, v_exp=v_exp, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kr, vr = kr.double().cpu().numpy(), vr.double().cpu().numpy()
    for i, s in enumerate(slots):
        for h in range(hkv):
            if s < 0:
                wk = wv = np.zeros(D)
            else:
                wk, wv = (x[s % B] for x in ref.tile_values(want[s // B, h], B, D, k_exp, v_exp))
            assert np.array_equal(kr[i, h], wk) and np.array_equal(vr[i, h], wv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,D", [(8, 64), (16, 128), (32, 128), (16, 64), (32, 64), (8, 128)])
def test_read_runs_of_tokens(dtype, B, D):
    """Whole runs in order, as a slot map gives them, over more tokens than a CTA holds, some
    of them unmapped."""
    dev = device()
    g = torch.Generator().manual_seed(5)
    hkv, pages = 3, 40
    pool, kv, vv = ref.make_pool(g, pages, hkv, B, D)
    order = torch.randperm(pages, generator=g)
    slot = (order[:, None] * B + torch.arange(B)).reshape(-1)[3:-5].clone()
    k, v = d2f.kv4_read(pool.to(dev), slot.to(dev), head_dim=D, block_size=B, dtype=dtype)
    pg, o = (slot // B).numpy(), (slot % B).numpy()
    assert np.array_equal(k.double().cpu().numpy(), kv[pg, :, o])
    assert np.array_equal(v.double().cpu().numpy(), vv[pg, :, o])
    gone = torch.rand(slot.shape, generator=g) < 0.2
    slot[gone] = -1
    k, v = d2f.kv4_read(pool.to(dev), slot.to(dev), head_dim=D, block_size=B, dtype=dtype)
    want = np.where(gone.numpy()[:, None, None], 0.0, kv[pg, :, o])
    assert np.array_equal(k.double().cpu().numpy(), want)
    want = np.where(gone.numpy()[:, None, None], 0.0, vv[pg, :, o])
    assert np.array_equal(v.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extremes(dtype):
    """Infinities saturate, a NaN makes its group NaN, small groups vanish, large ones clip."""
    dev = device()
    B, D = 16, 64
    x = torch.zeros((B, 1, D))
    x[0, 0, 0], x[0, 0, 1] = float("inf"), 1.0
    x[1, 0, 20] = float("-inf")
    x[2, 0, 40], x[2, 0, 41] = float("nan"), 2.0
    x[3, 0, :16] = 6 * 2.0 ** -11
    x[4, 0, :16] = 2.0 ** 20
    x[5, 0, 3] = 448 * 6.0
    x = x.to(dtype)
    pool = d2f.kv4_pool(dev, num_pages=1, num_heads_kv=1, head_dim=D, block_size=B)
    d2f.kv4_append(x.to(dev), x.to(dev), i32([0], dev), i32([0], dev), pool, block_size=B)
    k, v = d2f.kv4_read(pool, torch.arange(B, device=dev), head_dim=D, block_size=B, dtype=dtype)
    k, v = k.float().cpu(), v.float().cpu()
    assert torch.equal(torch.isnan(k), torch.isnan(v))
    assert torch.equal(torch.nan_to_num(k), torch.nan_to_num(v))
    k = k[:, 0]
    assert k[0, 0] == 2688 and k[0, 1] == 0 and k[1, 20] == -2688
    assert torch.isnan(k[2, 32:48]).all() and not torch.isnan(k[2, :32]).any()
    assert (k[3, :16] == 0).all() and (k[4, :16] == 2688).all() and k[5, 3] == 2688


def test_device_count_and_bad_entries():
    dev = device()
    g = torch.Generator().manual_seed(1)
    B, D, hkv = 16, 128, 2
    k = torch.randn((64, hkv, D), generator=g).to(torch.bfloat16)
    src, dst, m = [0, 16, 32, 48], [3, 1, 2, 0], [16, 16, 16, 16]
    for count, entries in ((2, 2), (9, 4), (-1, 0), (0, 0)):
        pool = d2f.kv4_pool(dev, num_pages=4, num_heads_kv=hkv, head_dim=D, block_size=B)
        d2f.kv4_append(k.to(dev), k.to(dev), i32(src, dev), i32(dst, dev), pool, block_size=B,
                       n_append_dev=i32([count], dev))
        want = expected_pool(k, k, list(zip(src, dst, m))[:entries], 4, B, D, 0, 0)
        assert np.array_equal(pool.cpu().numpy(), want)
    for bad in (dict(src=[49, 0]), dict(src=[-1, 0]), dict(dst=[4, 0]), dict(dst=[-1, 0]),
                dict(m=[17, 16]), dict(m=[-1, 16])):
        e = dict(src=[0, 16], dst=[1, 2], m=[16, 16])
        e.update(bad)
        pool = d2f.kv4_pool(dev, num_pages=4, num_heads_kv=hkv, head_dim=D, block_size=B)
        err = i32([0], dev)
        d2f.kv4_append(k.to(dev), k.to(dev), i32(e["src"], dev), i32(e["dst"], dev), pool,
                       block_size=B, n_rows=i32(e["m"], dev), err=err)
        torch.cuda.synchronize()
        assert int(err) == 4
        want = expected_pool(k, k, [(e["src"][1], e["dst"][1], e["m"][1])], 4, B, D, 0, 0)
        assert np.array_equal(pool.cpu().numpy(), want)
    err = i32([0], dev)
    pool = torch.full((4, hkv, B * D * 9 // 8), 0x31, dtype=torch.uint8, device=dev)
    kr, vr = d2f.kv4_read(pool, torch.tensor([64, -2, 5], device=dev), head_dim=D, block_size=B,
                          err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    assert (kr[:2] == 0).all() and (vr[:2] == 0).all() and (kr[2] != 0).any()

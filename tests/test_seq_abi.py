"""Host-side refusals of the prompt and token attention and of the token store (no GPU: every call
here is refused before anything is enqueued), and the tests' own 64-bit attention."""
import ctypes

import numpy as np
import pytest
import torch

import seq_ref as ref

from block_causal_kv_gb300 import d2f

P = ctypes.c_void_p(16)   # an aligned pointer that is never dereferenced
ODD = ctypes.c_void_p(8)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return d2f.load()


def msg(lib):
    return lib.d2f_last_error_string().decode()


def store(lib, k=P, v=P, slot=P, n=1, kp=P, vp=P, h=2, d=128, b=16, pages=4, dt=0):
    return lib.d2f_kv_store(k, v, slot, n, kp, vp, h, d, b, pages, dt, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(h=0), 1), (dict(d=0), 1), (dict(b=0), 1), (dict(pages=-1), 1),
    (dict(dt=2), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slot=None), 1), (dict(kp=None), 1),
    (dict(vp=None), 1), (dict(k=ODD), 1), (dict(kp=ODD), 1), (dict(n=2 ** 31 - 1, h=1 << 12), 2),
    (dict(d=1 << 21), 2), (dict(h=1 << 22), 2)])
def test_store_refusals(lib, kw, status):
    assert store(lib, **kw) == status and msg(lib)


def prompt(lib, q=P, k=P, v=P, start=P, kp=P, vp=P, table=P, maxp=8, ctx=P, out=P, batch=2, rows=40,
           max_ctx=64, hq=4, h=2, d=128, b=16, pages=4, dt=0, mb=1, scale=0.1, ws=P, wsb=1 << 40):
    return lib.d2f_prompt_attn(q, k, v, start, kp, vp, table, maxp, ctx, out, None, batch, rows, max_ctx,
                               hq, h, d, b, pages, dt, mb, ctypes.c_float(scale), ws, wsb, None, None)


def token(lib, q=P, kn=P, vn=P, kp=P, vp=P, table=P, maxp=8, ctx=P, out=P, batch=2, max_ctx=128, hq=4,
          h=2, d=128, b=16, pages=4, dt=0, scale=0.1, ws=P, wsb=1 << 40):
    return lib.d2f_token_attn(q, kn, vn, kp, vp, table, maxp, ctx, out, None, batch, max_ctx, hq, h, d, b,
                              pages, dt, ctypes.c_float(scale), ws, wsb, None, None)


SHARED = [(dict(batch=-1), 1), (dict(max_ctx=-1), 1), (dict(hq=3), 1), (dict(hq=0), 1), (dict(h=0), 1),
          (dict(dt=2), 1), (dict(b=0), 1), (dict(b=257), 2), (dict(d=96), 2), (dict(d=256), 2),
          (dict(batch=65536), 2), (dict(hq=65536), 2), (dict(scale=0.0), 1),
          (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(maxp=-1), 1),
          (dict(pages=-1), 1), (dict(max_ctx=129), 1), (dict(maxp=2 ** 28), 2), (dict(q=None), 1),
          (dict(out=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1),
          (dict(pages=0), 1), (dict(q=ODD), 1), (dict(kp=ODD), 1), (dict(out=ODD), 1)]


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(rows=-1), 1), (dict(rows=2 ** 30 + 1), 2), (dict(mb=-1), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(start=None), 1), (dict(ctx=None), 1), (dict(k=ODD), 1),
    (dict(rows=2 ** 30, hq=64, h=64), 2)])
def test_prompt_refusals(lib, kw, status, dt):
    assert prompt(lib, **dict(dict(dt=dt), **kw)) == status and msg(lib)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(kn=None), 1), (dict(vn=None), 1), (dict(ctx=None), 1), (dict(kn=ODD), 1),
    (dict(ws=None, max_ctx=16384, maxp=1024), 6), (dict(wsb=64, max_ctx=16384, maxp=1024), 6),
    (dict(ws=ODD, max_ctx=16384, maxp=1024), 1)])
def test_token_refusals(lib, kw, status, dt):
    # (without a GPU the plan counts one SM: one pair, so that it splits there too)
    one = dict(batch=1, hq=1, h=1) if "ws" in kw or "wsb" in kw else {}
    assert token(lib, **dict(dict(dt=dt, **one), **kw)) == status and msg(lib)


def test_nothing_to_do_is_ok(lib):
    assert store(lib, n=0, k=None) == 0
    assert prompt(lib, rows=0, q=None) == 0 and prompt(lib, batch=0, q=None) == 0
    assert token(lib, batch=0, q=None) == 0


def test_sizes(lib):
    # one request of many rows is not split; neither is a short one
    assert d2f.prompt_attn_workspace_size(1, 100000, 0, 32, 32, 128, 16) == 0
    assert d2f.prompt_attn_workspace_size(1, 64, 64, 4, 4, 64, 16, d2f.F32) == 0
    for fn in (lambda: d2f.prompt_attn_workspace_size(1, 16, 64, 5, 2, 128, 16),
               lambda: d2f.token_attn_workspace_size(1, 64, 5, 2, 128, 16)):
        with pytest.raises(d2f.D2FError) as e:
            fn()
        assert e.value.status == 1


def test_binding_checks_tensors():
    x = torch.zeros(16, 2, 128)
    i = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(4, 2, 16, 128)
    ws = torch.zeros(1)
    with pytest.raises(ValueError):       # not on a GPU
        d2f.prompt_attn(x, x, x, i, out=x, lse=x[..., 0].contiguous(), workspace=ws)
    with pytest.raises(ValueError):
        d2f.prompt_attn(x, x[:8], x, i, out=x, lse=x[..., 0].contiguous(), workspace=ws)
    with pytest.raises(ValueError):
        d2f.prompt_attn(x, x, x, i, ctx_len=i[:1], out=x, lse=x[..., 0].contiguous(), workspace=ws)
    with pytest.raises(ValueError):
        d2f.token_attn(x, pool, pool, i[None].repeat(16, 1), i, block_size=16, max_ctx=0, k_new=x)
    with pytest.raises(ValueError):
        d2f.kv_store(x, x, torch.zeros(16, dtype=torch.int64), pool, pool, block_size=8)


def test_reference_attention():
    """The tests' own attention against torch's softmax on dense keys."""
    for mb in (0, 1, 3):
        p = ref.problem([5, 0, 9], [7, 3, 0], hq=4, hkv=2, D=32, B=4, dtype=torch.float32, seed=mb,
                        mask_block=mb)
        out, lse, av, _, keys = ref.attention(p)
        for b, n in enumerate(p["new"]):
            r = int(p["start"][b])
            tok = torch.arange(p["ctx"][b])
            page = torch.from_numpy(p["table"][b]).long()[tok // 4]
            for h in range(4):
                k = torch.cat([p["k_pool"][page, h // 2, tok % 4], p["k"][r:r + n, h // 2]]).double()
                v = torch.cat([p["v_pool"][page, h // 2, tok % 4], p["v"][r:r + n, h // 2]]).double()
                x = p["q"][r:r + n, h].double() @ k.T * 32 ** -0.5
                for i in range(n):
                    for j in range(n):
                        if mb and j // mb > i // mb:
                            x[i, len(tok) + j] = float("-inf")
                assert np.allclose(out[r:r + n, h], x.softmax(-1) @ v, atol=1e-12)
                assert np.allclose(lse[r:r + n, h], x.logsumexp(-1), atol=1e-12)
                assert (av[r:r + n, h] + 1e-12 >= np.abs(out[r:r + n, h])).all()
                assert keys[r:r + n, h].tolist() == (~x.isinf()).sum(1).tolist()

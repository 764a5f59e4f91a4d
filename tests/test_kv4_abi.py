"""Host-side refusals of the 4-bit cache, page map and log-probability entry points (no GPU:
every call here is refused before anything is enqueued), and the format's own arithmetic."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as ref

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


def append(lib, k=P, v=P, src=P, dst=P, n=1, total=16, pool=P, h=2, d=128, b=16, pages=4, ke=0,
           ve=0, dt=0):
    return lib.d2f_kv4_append(k, v, src, dst, None, None, n, total, pool, h, d, b, pages, ke, ve,
                              dt, None, None)


def read(lib, pool=P, slot=P, n=1, k=P, v=P, h=2, d=128, b=16, pages=4, ke=0, ve=0, dt=0):
    return lib.d2f_kv4_read(pool, slot, n, k, v, h, d, b, pages, ke, ve, dt, None, None)


SIZES = [(dict(h=0), 1), (dict(pages=-1), 1), (dict(dt=2), 1), (dict(dt=-1), 1), (dict(ke=65), 1),
         (dict(ve=-65), 1), (dict(d=96), 2), (dict(d=256), 2), (dict(b=4), 2), (dict(b=64), 2),
         (dict(b=0), 2), (dict(n=-1), 1)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(total=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(src=None), 1),
    (dict(dst=None), 1), (dict(pool=None), 1), (dict(k=ODD), 1), (dict(v=ODD), 1),
    (dict(pool=ODD), 1), (dict(n=2 ** 30, h=4), 2)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status and msg(lib)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(pool=None), 1), (dict(slot=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=ODD), 1), (dict(v=ODD), 1), (dict(pool=ODD), 1), (dict(n=2 ** 31 - 1, h=64), 2)])
def test_read_refusals(lib, kw, status):
    assert read(lib, **kw) == status and msg(lib)


def attention(lib, q=P, kw=P, vw=P, pool=P, table=P, maxp=8, ctx=P, qs=P, out=P, batch=1, total=16,
              max_q=16, max_ctx=64, hq=4, h=2, d=128, b=16, pages=4, ke=0, ve=0, dt=1, scale=0.1,
              ws=P, wsb=1 << 40):
    return lib.d2f_block_attn_kv4(q, kw, vw, pool, table, maxp, ctx, qs, out, None, batch, total,
                                  max_q, max_ctx, hq, h, d, b, pages, ke, ve, dt,
                                  ctypes.c_float(scale), ws, wsb, None, None)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("kw,status", [x for x in SIZES if "n" not in x[0] and "dt" not in x[0]] + [
    (dict(hq=3), 1), (dict(hq=0), 1), (dict(batch=-1), 1), (dict(max_q=17), 1),
    (dict(max_ctx=-1), 1), (dict(max_ctx=129), 1), (dict(maxp=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(kw=None), 1), (dict(vw=None), 1),
    (dict(out=None), 1), (dict(ctx=None), 1), (dict(qs=None), 1), (dict(pool=None), 1),
    (dict(table=None), 1), (dict(q=ODD), 1), (dict(pool=ODD), 1), (dict(out=ODD), 1),
    (dict(batch=40000), 2), (dict(ws=None), 6), (dict(wsb=1), 6)])
def test_attention_refusals(lib, kw, status, dt):
    assert attention(lib, dt=dt, **kw) == status and msg(lib)


def test_attention_refuses_other_dtypes(lib):
    assert attention(lib, dt=2) == 1


@pytest.mark.parametrize("dt", [0, 1])
def test_attention_refuses_page_tables_past_32_bits(lib, dt):
    assert attention(lib, dt=dt, maxp=2 ** 27) == 2 and "max_pages_per_seq" in msg(lib)


@pytest.mark.parametrize("kw", [
    dict(batch=1025, total=1025 * 16),                        # sequences on tensor cores
    dict(total=2 ** 24, max_q=2 ** 24, h=256, hq=256),        # rows of one sequence x its keys
    dict(maxp=2 ** 26, total=2 ** 16, max_q=2 ** 16, h=4, hq=4)])
def test_attention_size_limits_of_the_tensor_core_path(lib, kw):
    assert attention(lib, dt=0, **kw) == 2 and msg(lib)


def page_map(lib, batch=2, b=16, maxp=4, cap=32, app=2, null=()):
    ptr = [None if i in null else P for i in range(14)]
    return lib.d2f_page_map(batch, b, maxp, cap, app, *ptr, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(b=0), 1), (dict(maxp=-1), 1), (dict(cap=-1), 1), (dict(app=-1), 1),
    (dict(batch=16385), 2)] + [(dict(null=(i,)), 1) for i in range(14)])
def test_page_map_refusals(lib, kw, status):
    assert page_map(lib, **kw) == status and msg(lib)


def logprobs(lib, logits=P, stride=1000, dt=0, vocab=1000, rows=4, tokens=P, n=4, k=2, lp=P, ids=P,
             tlp=P, ws=P, wsb=1 << 40):
    return lib.d2f_token_logprobs(logits, stride, dt, vocab, rows, None, tokens, n, k, lp, None, ids,
                                  tlp, ws, wsb, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(vocab=0), 1), (dict(k=-1), 1), (dict(vocab=10, k=11), 1), (dict(k=33), 2),
    (dict(dt=2), 1), (dict(n=65536), 2), (dict(vocab=2 ** 30 + 1), 2), (dict(stride=999), 1),
    (dict(rows=0), 1), (dict(logits=None), 1), (dict(tokens=None), 1), (dict(lp=None), 1),
    (dict(ids=None), 1), (dict(tlp=None), 1)])
def test_logprobs_refusals(lib, kw, status):
    assert logprobs(lib, **kw) == status and msg(lib)


def test_nothing_to_do_is_ok(lib):
    assert append(lib, n=0, k=None) == 0
    assert read(lib, n=0, slot=None) == 0
    assert logprobs(lib, n=0, logits=None) == 0
    assert attention(lib, batch=0, total=0, max_q=0) == 0


def test_sizes(lib):
    assert d2f.kv4_page_bytes(128, 16) == 2304 and d2f.kv4_page_bytes(64, 8) == 576
    for bad in ((96, 16), (128, 12)):
        with pytest.raises(d2f.D2FError) as e:
            d2f.kv4_page_bytes(*bad)
        assert e.value.status == 2
    with pytest.raises(d2f.D2FError) as e:
        d2f.attn_kv4_workspace_size(1, 16, 16, 64, 5, 2, 128, 16)
    assert e.value.status == 1
    with pytest.raises(d2f.D2FError) as e:
        d2f.logprobs_workspace_size(4, 1000, 40)
    assert e.value.status == 2


def test_binding_checks_tensors():
    x = torch.zeros(16, 2, 128)
    i = torch.zeros(1, dtype=torch.int32)
    pool = torch.zeros(4, 2, 2304, dtype=torch.uint8)
    with pytest.raises(ValueError):
        d2f.kv4_append(x, x, i, i, pool[:, :, :2000], block_size=16)
    with pytest.raises(ValueError):
        d2f.kv4_append(x, x[:8], i, i, pool, block_size=16)
    with pytest.raises(ValueError):       # not on a GPU
        d2f.kv4_append(x, x, i, i, pool, block_size=16)
    with pytest.raises(ValueError):
        d2f.kv4_read(pool[:, :1], torch.zeros(2, dtype=torch.int64), head_dim=64, block_size=16)
    with pytest.raises(ValueError):
        d2f.token_logprobs(x[0], i)
    with pytest.raises(ValueError):
        d2f.page_map(i, i, i, i, i, block_size=16, capacity=4, max_append=1)


def test_reference_format_round_trip():
    """The tests' own encoder and byte layouts agree with one another."""
    g = torch.Generator().manual_seed(0)
    pool, k, v = ref.make_pool(g, 3, 2, 16, 64, 1, -2)
    for p in range(3):
        for h in range(2):
            tk, tv = ref.tile_values(pool[p, h].numpy(), 16, 64, 1, -2)
            assert np.array_equal(tk, k[p, h]) and np.array_equal(tv, v[p, h])
    # hand-worked group: scale e4m3(6 / 6) = 1, codes to the nearest, ties to even
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.3, -0.2, 2.6, 5.1, 0, 1, 3, 4]])
    codes, bits, val = ref.encode(x, 0)
    assert bits.tolist() == [[56]]
    assert val[0].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -0.0, 3, 6, 0, 1, 3, 4]
    assert codes[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 8, 5, 7, 0, 2, 5, 6]

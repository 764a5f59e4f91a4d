"""d2f_page_map against a request-by-request form."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def case(seed, batch, B, longest, *, cached=0, free_share=1.1, table_slack=1, extra_rows=5,
         extra_app=3, zeros=False):
    g = np.random.default_rng(seed)
    new = g.integers(0 if zeros else 1, longest + 1, batch)
    if zeros and batch > 2:
        new[0] = new[-1] = new[batch // 2] = 0
    ctx = g.integers(0, cached + 1, batch) * B
    need = -(-new // B)
    per = max(1, int((ctx // B + need).max()) + table_slack)
    free = int(need.sum() * free_share)
    pages = g.permutation(free + 50)
    return dict(new=new.tolist(), ctx=ctx.tolist(), table=np.full((batch, per), -7, np.int32),
                free=pages.astype(np.int32), count=free, B=B, capacity=int(new.sum()) + extra_rows,
                max_append=max(0, int(need.sum()) + extra_app))


def run(c, dev, err=None, in_place=False):
    t = [i32(c["new"], dev), i32(c["ctx"], dev), torch.from_numpy(c["table"].copy()).to(dev),
         torch.from_numpy(c["free"]).to(dev), i32([c["count"]], dev)]
    kw = dict(ctx_len_out=t[1], free_count_out=t[4]) if in_place else {}
    return d2f.page_map(*t, block_size=c["B"], capacity=c["capacity"], max_append=c["max_append"],
                        err=err, **kw)


def check(c, r):
    w = ref.page_map(c["new"], c["ctx"], c["table"], c["free"], c["count"], c["B"], c["capacity"],
                     c["max_append"])
    for key, name in (("ctx_len", "ctx_len"), ("row_start", "row_start"), ("admitted", "admitted"),
                      ("slot", "slot"), ("app_src", "src"), ("app_dst", "dst"),
                      ("app_rows", "rows")):
        assert r[key].cpu().tolist() == list(w[name]), key
    assert np.array_equal(r["page_table"].cpu().numpy(), w["table"])
    assert int(r["n_append"]) == w["n_append"] and int(r["free_count"]) == w["free_count"]
    return w


CASES = [
    dict(seed=1, batch=1, B=16, longest=1), dict(seed=2, batch=1, B=16, longest=500),
    dict(seed=3, batch=16, B=16, longest=512), dict(seed=4, batch=33, B=8, longest=70, zeros=True),
    dict(seed=5, batch=7, B=32, longest=100, cached=5),
    dict(seed=6, batch=40, B=16, longest=90, cached=3, free_share=0.5, zeros=True),
    dict(seed=7, batch=20, B=16, longest=60, free_share=0.0),
    dict(seed=8, batch=30, B=16, longest=200, cached=6, table_slack=-4),
    dict(seed=9, batch=25, B=1, longest=9, zeros=True), dict(seed=10, batch=25, B=5, longest=31),
    dict(seed=11, batch=12, B=16, longest=99, extra_app=-10),
    dict(seed=12, batch=3000, B=16, longest=40, zeros=True, free_share=0.9),
    dict(seed=13, batch=300, B=16, longest=900, cached=9, free_share=0.8),
    dict(seed=14, batch=2, B=16, longest=60000),
    dict(seed=15, batch=16384, B=8, longest=3, zeros=True),
    dict(seed=16, batch=700, B=32, longest=1500, cached=9, table_slack=-6, extra_rows=0,
         extra_app=0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kw", CASES, ids=lambda k: "seed%d" % k["seed"])
def test_page_map(kw, in_place):
    dev = device()
    c = case(**kw)
    err = i32([0], dev)
    r = run(c, dev, err, in_place)
    torch.cuda.synchronize()
    w = check(c, r)
    assert int(err) == (0 if all(w["admitted"]) else 7)


def test_empty_batch_and_no_tokens():
    dev = device()
    r = d2f.page_map(i32([], dev), i32([], dev), torch.zeros((0, 4), dtype=torch.int32, device=dev),
                     i32([3], dev), i32([1], dev), block_size=16, capacity=4, max_append=2)
    assert r["row_start"].tolist() == [0] and r["slot"].tolist() == [-1] * 4
    assert int(r["n_append"]) == 0 and int(r["free_count"]) == 1
    c = dict(new=[0, 0], ctx=[16, 0], table=np.full((2, 2), -7, np.int32),
             free=np.array([5], np.int32), count=1, B=16, capacity=0, max_append=0)
    check(c, run(c, dev))


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("change", [dict(new=[3, -1, 4]), dict(ctx=[0, 16, 7]),
                                    dict(ctx=[0, -16, 16]), dict(count=-1), dict(capacity=11)])
def test_inconsistent_states_write_nothing(change, big):
    dev = device()
    c = dict(new=[3, 5, 4], ctx=[0, 16, 16], table=np.full((3, 4), -7, np.int32),
             free=np.arange(20, dtype=np.int32), count=9, B=16, capacity=300000 if big else 12,
             max_append=8)
    if big and "capacity" in change:
        change = dict(new=[299990, 5, 6])
    c.update(change)
    err = i32([0], dev)
    t = [i32(c["new"], dev), i32(c["ctx"], dev), torch.from_numpy(c["table"]).to(dev),
         torch.from_numpy(c["free"]).to(dev), i32([c["count"]], dev)]
    ctx_out, free_out = i32([-9] * 3, dev), i32([-9], dev)
    r = d2f.page_map(*t, block_size=16, capacity=c["capacity"], max_append=8, ctx_len_out=ctx_out,
                     free_count_out=free_out, err=err)
    torch.cuda.synchronize()
    assert int(err) == 1
    assert ctx_out.tolist() == [-9] * 3 and int(free_out) == -9
    assert (r["page_table"] == -7).all()


@pytest.mark.parametrize("capacity", [32, 300000])
def test_replays_from_a_graph(capacity):
    """In place, captured: every replay takes the next pages."""
    dev = device()
    new, ctx = i32([20, 5], dev), i32([0, 16], dev)
    table = torch.full((2, 8), -1, dtype=torch.int32, device=dev)
    free, count = i32(list(range(30)), dev), i32([30], dev)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = d2f.page_map(new, ctx, table, free, count, block_size=16, capacity=capacity,
                             max_append=4, free_count_out=count)
        for k in range(3):
            g.replay()
            s.synchronize()
            assert int(count) == 30 - 3 * (k + 1)
            top = 29 - 3 * k
            assert r["app_dst"].tolist() == [top, top - 1, top - 2, -1]
            slot = r["slot"][:26].tolist()
            assert slot == ([top * 16 + i for i in range(16)] +
                            [(top - 1) * 16 + i for i in range(4)] +
                            [(top - 2) * 16 + i for i in range(5)] + [-1])

"""d2f_page_map over a batch whose contexts it made itself, and after calls that it refused."""
import numpy as np
import pytest
import torch

from gpu_common import device
from test_gpu_page_map import check, i32

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("capacity", [600, 300000])
def test_contexts_that_end_inside_a_page_stay_in_the_batch(capacity, in_place):
    """Prompts of any length, then new requests in other slots while the first ones wait with
    nothing new."""
    dev = device()
    B = 16
    table = np.full((6, 20), -7, np.int32)
    free = np.random.default_rng(1).permutation(90).astype(np.int32)
    c = dict(new=[251, 0, 17, 0, 16, 0], ctx=[0] * 6, table=table, free=free, count=90, B=B,
             capacity=capacity, max_append=60)
    t = [i32(c["new"], dev), i32(c["ctx"], dev), torch.from_numpy(table.copy()).to(dev),
         torch.from_numpy(free).to(dev), i32([90], dev)]

    def call():
        kw = dict(ctx_len_out=t[1], free_count_out=t[4]) if in_place else {}
        err = i32([0], dev)
        r = d2f.page_map(*t, block_size=B, capacity=c["capacity"], max_append=c["max_append"],
                         err=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        return r
    first = check(c, call())
    assert first["ctx_len"] == [251, 0, 17, 0, 16, 0]
    c.update(new=[0, 33, 0, 1, 40, 0], ctx=first["ctx_len"], table=first["table"],
             count=first["free_count"])
    t[0] = i32(c["new"], dev)
    t[1], t[4] = i32(c["ctx"], dev), i32([c["count"]], dev)
    second = check(c, call())
    assert second["admitted"] == [1] * 6 and second["ctx_len"] == [251, 33, 17, 1, 56, 0]


@pytest.mark.parametrize("capacity", [12, 300000])
@pytest.mark.parametrize("change", [dict(new=[3, -1, 4]), dict(ctx=[0, 16, 7]),
                                    dict(ctx=[0, -16, 16]), dict(count=-1), dict(new=[299990, 9, 4])])
@pytest.mark.parametrize("given", [(), ("ctx_len_out",), ("free_count_out",),
                                   ("ctx_len_out", "free_count_out")])
def test_results_of_a_refused_state_are_an_empty_map(change, capacity, given):
    """Every result that the call makes is written: no rows, no pages, the contexts and the free
    count as they were."""
    dev = device()
    c = dict(new=[3, 5, 4], ctx=[0, 16, 16], count=9)
    c.update(change)
    table = torch.full((3, 4), -7, dtype=torch.int32, device=dev)
    free = torch.arange(20, dtype=torch.int32, device=dev)
    new, ctx, count, err = i32(c["new"], dev), i32(c["ctx"], dev), i32([c["count"]], dev), i32([0], dev)
    out = dict(ctx_len_out=ctx.clone(), free_count_out=count.clone())
    # memory that the results may come from, full of other numbers
    dirty = [torch.full((n,), 9, dtype=t, device=dev) for _ in range(16)
             for n, t in ((3 + 1 + 4 + 1 + 24, torch.int32), (3, torch.uint8), (capacity, torch.int64))]
    torch.cuda.synchronize()
    del dirty
    r = d2f.page_map(new, ctx, table, free, count, block_size=16, capacity=capacity, max_append=8,
                     err=err, **{k: out[k] for k in given})
    torch.cuda.synchronize()
    assert int(err) == 1 and int(r["n_append"]) == -1 and (table == -7).all()
    assert r["ctx_len"].tolist() == c["ctx"] and r["free_count"].tolist() == [c["count"]]
    assert r["row_start"].tolist() == [0] * 4 and r["admitted"].tolist() == [0] * 3
    assert (r["slot"] == -1).all() and r["slot"].numel() == capacity
    assert r["app_src"].tolist() == [-1] * 8 and r["app_dst"].tolist() == [-1] * 8
    assert r["app_rows"].tolist() == [0] * 8

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

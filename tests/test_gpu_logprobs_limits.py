"""d2f_token_logprobs at the largest vocabularies."""
import math

import pytest
import torch

from gpu_common import device

from block_causal_kv_gb300 import d2f

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 2 ** 30), (torch.float32, 2 ** 29 + 3)])
def test_rows_masked_with_the_lowest_value(dtype, V):
    """Hundreds of millions of logits at the type's lowest value beside one that is not: it has
    all the probability, and the entropy is 0."""
    dev = device()
    low = torch.finfo(dtype).min
    x = torch.full((1, V), low, dtype=dtype, device=dev)
    at = V - 7
    x[0, at] = 2.5
    r = d2f.token_logprobs(x, torch.tensor([at], dtype=torch.int32, device=dev), top_k=3)
    assert r["logprob"].tolist() == [0.0] and r["entropy"].tolist() == [0.0]
    assert r["top_id"].tolist() == [[at, 0, 1]] and float(r["top_logprob"][0, 0]) == 0.0
    # all alike: the sums stay exact, ln V has a rounding of its own
    x[0, at] = low
    r = d2f.token_logprobs(x, torch.tensor([at], dtype=torch.int32, device=dev), top_k=3)
    assert abs(float(r["entropy"]) - math.log(V)) <= 2.0 ** -20 * math.log(V)
    assert abs(float(r["logprob"]) + math.log(V)) <= 2.0 ** -20 * math.log(V)
    assert r["top_id"].tolist() == [[0, 1, 2]]

"""Refusals of the binding of the prompt attention (no GPU)."""
import pytest
import torch

from block_causal_kv_gb300 import d2f


@pytest.mark.parametrize("given", [("k_pool",), ("v_pool",), ("page_table",),
                                   ("k_pool", "v_pool", "page_table")])
def test_a_cached_prefix_without_its_lengths_is_refused(given):
    """Pools or a page table without ctx_len would be a prompt without its prefix."""
    x = torch.zeros(16, 2, 128)
    pool = torch.zeros(4, 2, 16, 128)
    have = dict(k_pool=pool, v_pool=pool, page_table=torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(ValueError, match="ctx_len"):
        d2f.prompt_attn(x, x, x, torch.tensor([0, 16], dtype=torch.int32), out=x, want_lse=False,
                        workspace=torch.zeros(1), **{n: have[n] for n in given})

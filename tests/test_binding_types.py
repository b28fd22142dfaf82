"""Arguments that are no tensors, or tensors of the wrong rank, are TypeErrors and ValueErrors of
the binding that name the argument (no GPU: CPU tensors are refused the same way)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import api

NO_TENSORS = [None, [[1.0]], np.zeros((2, 4, 2, 8), np.float32)]


@pytest.mark.parametrize("bad", NO_TENSORS, ids=["none", "list", "numpy"])
def test_pools_that_are_no_tensors(bad):
    q = torch.zeros(2, 4, 8, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="k_cache"):
        tl.tl_paged_attn_decode(q, bad, bad, table, lens, 1.0)
    with pytest.raises(TypeError, match="k_cache"):
        tl.tl_paged_attn_prefill(q[:, None], bad, bad, table, lens[:, None], 1.0)
    with pytest.raises(TypeError, match="k_cache"):
        tl.tl_paged_attn_decode_write_rope(q, q, q, lens.long(), lens, lens.long(), bad, bad, table,
                                           lens, 1.0)


@pytest.mark.parametrize("bad", NO_TENSORS + [torch.zeros(4, dtype=torch.int64)],
                         ids=["none", "list", "numpy", "cpu"])
def test_rotary_tables_that_are_no_tensors(bad):
    with pytest.raises(TypeError, match="freqs"):
        api._need_table_of_turns(bad, 8, torch.device("cuda", 0))


def test_pools_of_the_wrong_rank(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    dev, pool = torch.device("cuda", 0), torch.zeros(2, 4, 2, 8)
    assert api._need_pools(pool, pool, dev) == pool.shape
    for k, v in ((pool[0], pool[0]), (pool, pool[0]), (pool, pool[:1])):
        with pytest.raises(ValueError):
            api._need_pools(k, v, dev)
    with pytest.raises(TypeError):
        api._need_pools(pool, pool, dev, torch.int8)
    with pytest.raises(TypeError):
        api._need_pools(pool, pool.double(), dev)

"""KV4Cache and trees of drafted tokens without a GPU: nodes need a tree that has begun."""
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests.test_kv4_cpu import lib  # noqa: F401


def test_nodes_before_start_tree_are_refused(lib):  # noqa: F811
    cache = q.KV4Cache(q.make_kv4_config(2, page_size=16), 1, 4, device="cpu")
    x, cu, mask = torch.zeros(1, 2, 128, dtype=torch.bfloat16), torch.tensor([0, 1], dtype=torch.int32), torch.ones(1, dtype=torch.int64)
    ints = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: cache.append(x, x, cu, 1, tree_mask=mask), lambda: cache.attend(x, 0.1, cu_q=cu, tree_mask=mask),
                 lambda: cache.keep(ints, ints[0])):
        with pytest.raises(q.QCacheError, match="start_tree"):
            call()
    with pytest.raises(ValueError, match="causal"):
        cache.attend(x, 0.1, cu_q=cu, tree_mask=mask, causal=False)
    # rows that are no nodes, and nodes whose base is given, go on to the library (which wants a GPU)
    for call in (lambda: cache.append(x, x, cu, 1), lambda: cache.append(x, x, cu, 1, tree_mask=mask, tree_base=ints[0])):
        with pytest.raises(q.QCacheError, match="CUDA"):
            call()

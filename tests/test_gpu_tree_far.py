"""Trees in large memory: rows of probabilities beyond 2^31 elements, pages beyond 2^32 bytes; and single nodes without offsets."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import tree_ref as tr
from tests.test_gpu_kv4 import error_word, ints
from tests.test_gpu_tree import Tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,max_rows", [(torch.float32, 3), (torch.bfloat16, 3), (torch.bfloat16, 9)])
def test_rows_beyond_31_bits(dtype, max_rows):
    """Sequences at the start and the end of an array of more than 2^31 elements; those between have no rows."""
    V, n = 100003, 3
    rows = 2 ** 31 // V + 40
    x = torch.zeros(rows, V, dtype=dtype, device="cuda")
    best = [7, 99991, 50000]
    for k, token in enumerate(best):
        x[k, token] = x[rows - n + k, token] = 1
    tokens = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    for r in (0, rows - n):
        tokens[r + 1:r + 3] = ints(best[:2])
    cu = ints([0, n, rows - n, rows])  # the one between has too many rows
    kept, new, count, err = ints(np.zeros((3, max_rows))), ints(np.zeros((3, max_rows))), ints([0] * 3), error_word()
    for way in range(2 if dtype == torch.float32 else 1):
        new.zero_(), err.zero_()
        if way == 0:
            q.mla_qcache_verify_greedy(x, tokens, cu, max_rows, kept, new, count, err)
        else:
            u = torch.full((rows,), 0.5, device="cuda")
            q.mla_qcache_verify_sampled(x, tokens, cu, max_rows, u, u[:3], kept, new, count, err, draft_probs=x)
        torch.cuda.synchronize()
        assert count.tolist() == [3, 0, 3] and int(err) == q.DEV_ROWS
        for b in (0, 2):
            assert new[b, :3].tolist() == best and kept[b, :3].tolist() == [0, 1, 2]


def test_pages_beyond_32_bits():
    """A pool of more than 2^32 bytes: attention and keeping read and move tokens at its end."""
    small = Tree([150, 90], [9, 9], Hkv=8, G=4, D=128, P=64, seed=3)
    want, wl = small.run()
    far = 2 ** 32 // small.pool.shape[1] + 10
    pool = torch.zeros(far + small.n_pages, small.pool.shape[1], dtype=torch.uint8, device="cuda")
    pool[far:] = small.pool
    near, table = small.pool, small.table.copy()
    small.pool, small.n_pages = pool, len(pool)
    out, lse = small.run(table=np.where(table < 10 ** 6, table + far, table))
    torch.cuda.synchronize()
    assert int(small.err) == 0 and torch.equal(out, want) and torch.equal(lse, wl)
    kept, count = np.array([[0, 2, 5, 8], [0, 1, 7, -1]]), [4, 3]
    expect = near.cpu().numpy().copy()
    for b in range(2):
        tr.keep(expect, table[b], small.base[b], kept[b, :count[b]], 8, 128, 128, 64)
    lens = ints(small.lens)
    q.mla_qcache_kv4_keep(small.cfg, ints(kept), ints(count), ints(small.base), ints(table + far), pool, lens, small.err)
    torch.cuda.synchronize()
    assert int(small.err) == 0 and lens.tolist() == [a + c for a, c in zip(small.base, count)]
    assert np.array_equal(pool[far:].cpu().numpy(), expect) and not pool[:far].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("base", [True, False])
def test_one_node_of_each_tree_without_offsets(dtype, base):
    """The newest node of each tree alone, and no offsets: without bases each is the whole of its tree."""
    c = Tree([120, 33, 9], [9, 9, 9], new=[1, 1, 1], Hkv=2, G=4, P=16, dtype=dtype, seed=5)
    if not base:
        c.base, c.masks = [T - 1 for T in c.lens], [[1]] * 3
    out, lse = torch.zeros(3, c.Hq, c.D, dtype=c.t, device="cuda"), torch.zeros(3, c.Hq, device="cuda")
    mask = tr.mask_tensor([m for ms in c.masks for m in ms], 1)[:, 0].contiguous()
    q.mla_qcache_kv4_attn_tree(c.cfg, c.q, mask, None, 1, ints(c.table), ints(c.lens), c.pool, c.D ** -0.5, out, c.workspace(1), c.err,
                               tree_base=ints(c.base) if base else None, lse=lse)
    same, sl = c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.compare(out, lse)
    assert torch.equal(out, same) and torch.equal(lse, sl)

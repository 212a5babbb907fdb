"""FP16 outputs over long contexts, where values average out: what is left of them is as exact as its own rounding and that of the
weights allow. Sums of many products on one side of zero would not be (the tensor cores' float32 sums round towards zero).

The bound goes by root mean squares: roundings are spread evenly and independent of one another, an output's own at most 2^-11 of it, a
weight's 2^-11 of it times the distance of its token's code from 7.5; each is 1 / sqrt(3) of that in the mean, taken together over some
ten thousand numbers, and a twentieth more."""
import math

import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import kv4_ref as ref, tree_ref as tr
from tests.test_gpu_kv4 import error_word, ints

pytestmark = pytest.mark.gpu


def cache(B, T, D, group, P, seed):
    """One kv head: random codes, values about zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cfg = q.make_kv4_config(1, D, group=group, page_size=P)
    pages = -(-T // P)
    pool = torch.randint(0, 256, (B * pages, q.kv4_page_bytes(cfg)), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((B * pages, P, D // group, 2), generator=g, device="cuda") * 0.1 + 0.2).half()
    numbers = torch.stack([scale[..., 0], -7.5 * scale[..., 0], scale[..., 1], -7.5 * scale[..., 1]], -1)
    pool[:, P * D:] = numbers.contiguous().view(torch.uint8).view(B * pages, -1)
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    return cfg, pool, table, g


def values(pool, pages, T, D, group, P):
    """Keys, values and the values' distance from the middle of their levels [T, D] in 64 bits."""
    r = pool[pages.long()]
    num = r[:, P * D:].contiguous().view(torch.float16).double().view(-1, D // group, 4)[:T].repeat_interleave(group, 1)

    def codes(first, nibble):
        at = torch.tensor([nibble(c, D) for c in range(D)], device="cuda")
        rows = r[:, first:first + P * D // 2].reshape(-1, D // 2)[:T]
        return (rows[:, at // 2] >> (4 * (at % 2)).to(torch.uint8) & 15).double()
    n = codes(P * D // 2, ref.value_nibble)
    return codes(0, ref.key_nibble) * num[..., 0] + num[..., 1], n * num[..., 2] + num[..., 3], (n - 7.5) * num[..., 2]


@pytest.mark.parametrize("D,group,B,T", [(128, 128, 16, 60000), (64, 32, 16, 60000), (128, 32, 4, 65000), (128, 64, 40, 9000)])
@pytest.mark.parametrize("rows,G,tree", [(1, 8, False), (4, 8, False), (4, 8, True), (1, 16, True), (6, 8, True)])
def test_outputs_over_long_contexts(D, group, B, T, rows, G, tree):
    P = 128
    cfg, pool, table, g = cache(B, T, D, group, P, D + group + rows)
    n, scale = B * rows, 1 / math.sqrt(D)
    qq = (torch.randn(n, G, D, generator=g, device="cuda") * 0.8).half()
    out, err = torch.empty_like(qq), error_word()
    cu, lens = ints([rows * b for b in range(B + 1)]), ints([T] * B)
    ws = torch.zeros(q.kv4_workspace_bytes(cfg, B, G, rows, table.shape[1]), dtype=torch.uint8, device="cuda")
    if tree:  # siblings under the tokens before the tree
        q.mla_qcache_kv4_attn_tree(cfg, qq, tr.mask_tensor([1 << i for i in range(rows)] * B, 1), cu, rows, table, lens, pool, scale, out, ws, err)
    else:
        q.mla_qcache_kv4_attn(cfg, qq, table, lens, pool, scale, out, ws, err, cu_q=cu, max_q=rows)
    torch.cuda.synchronize()
    assert int(err) == 0
    off = bound = mean = size = 0.0
    for b in range(B):
        k, v, far = values(pool, table[b], T, D, group, P)
        s = (qq[rows * b:rows * b + rows].double().reshape(rows * G, D) @ k.T).mul_(scale).view(rows, G, T)
        for i in range(rows):
            if tree:
                s[i, :, T - rows:T - rows + i] = -math.inf
            s[i, :, T - rows + i + 1:] = -math.inf
        p = torch.softmax(s.view(rows * G, T), -1)
        want, got = p @ v, out[rows * b:rows * b + rows].double().view(rows * G, D)
        off += float(((got - want) ** 2).sum())
        bound += float(((want ** 2).sum() + ((p ** 2) @ (far ** 2)).sum()) * 2.0 ** -22 / 3)
        mean += float((got - want).sum())
        size += float(want.abs().sum())
    assert math.sqrt(off) <= 1.05 * math.sqrt(bound), math.sqrt(off / bound)
    # Roundings on both sides of zero: the mean lies within six of its standard deviations. Above 32 rows it is values that are rounded, by
    # as little as weights are below, and all rows of a sequence share them: N errors that are the same have a sum of N times one in place
    # of sqrt(N) times, so that the standard deviation is up to sqrt(rows) times as large.
    shared = rows * G if rows * G > 32 else 1
    assert abs(mean) <= 6 * math.sqrt(shared * bound) and size > 0, (mean / size, mean / math.sqrt(bound))

"""Trees with FP16 outputs above 32 rows: weights enter in two FP16 parts. Values that FP16 holds exactly and scores near zero leave the
weights' rounding and the output's own as the only ones that show, so that a second part that is missing, or beside the wrong
token, lies outside the bound.

Bound of an output, from the arithmetic: scores s off by 2 D 2^-24 |q|.|k| (float32 sums; keys are exact), exponentials and their sums by
2^-20 and a 2^-24 for each token that counts, both in numerator and denominator; a weight's two parts leave 2^-22 of it, and 2^-32 of
the largest; the products are summed in float32, a step of 2^-23 for each of the two parts of a token that counts; joining and rescaling
2^-20. Tokens of a weight below 2^-50 do not count. Rounded once to FP16."""
import math

import numpy as np
import pytest
import torch

from tests import kv4_ref as ref, tree_ref as tr
from tests.test_gpu_tree import Tree

pytestmark = pytest.mark.gpu
FAR = -2400.0  # a far token's key: its weight is below 2^-50


def prepared(lens, sizes, near, wide, Hkv, G, D, group, P=16, seed=0):
    """A case whose values are (code - 7.5) 2^k, whose queries look at channel 0 alone, and which sees `near` of the tokens before
    each tree (spread over them), the others being far."""
    c = Tree(lens, sizes, Hkv=Hkv, G=G, D=D, group=group, P=P, dtype="fp16", seed=seed)
    rng = np.random.default_rng(seed + 1)
    pool = c.pool.cpu().numpy().copy()
    NG = D // group
    num = pool.reshape(len(pool), Hkv, -1)[:, :, P * D:].copy().view(np.float16).reshape(len(pool), Hkv, P, NG, 4)
    for b, (T, base) in enumerate(zip(lens, c.base)):
        t = np.arange(T)
        at = (c.table[b, t // P], slice(None), t % P)
        vs = 2.0 ** rng.integers(-1, 2, (T, Hkv, NG))
        num[(*at, slice(None), 2)], num[(*at, slice(None), 3)] = vs, -7.5 * vs
        far = np.ones(T, bool)
        far[base:] = False
        far[rng.permutation(base)[:near]] = False
        t = np.flatnonzero(far)
        at = (c.table[b, t // P], slice(None), t % P)
        num[(*at, slice(None), 0)], num[(*at, slice(None), 1)] = 0, FAR
    pool.reshape(len(pool), Hkv, -1)[:, :, P * D:] = num.reshape(len(pool), Hkv, -1).view(np.uint8)
    c.pool = torch.tensor(pool).cuda()
    qq = torch.zeros_like(c.q)
    qq[..., 0] = torch.tensor(rng.uniform(0.9, 1.1, qq.shape[:2]) * 0.0175 * math.sqrt(D), dtype=torch.float32).half().cuda()
    c.q = qq
    if wide:  # room for more: items are cut over the CTAs
        c.table = np.ascontiguousarray(np.concatenate([c.table, np.full((len(lens), 2 ** 20 // P), 10 ** 6, np.int32)], 1))
    return c


def statement(q, k, v, scale, ok):
    """(output, its bound, the output with weights in one part, with the second parts one token off) of one sequence."""
    n, Hq, D = q.shape
    G, half = Hq // k.shape[0], 2.0 ** -11
    out, bound, one, off = (np.zeros((n, Hq, D)) for _ in range(4))
    for h in range(Hq):
        kk, vv = k[h // G], v[h // G]
        s = (q[:, h] @ kk.T) * scale
        mag = (np.abs(q[:, h]) @ np.abs(kk).T) * abs(scale)
        for i in range(n):
            m = np.flatnonzero(ok[i])
            if not len(m):
                continue
            w = np.exp(s[i, m] - s[i, m].max())
            counts = w > 2.0 ** -50
            lost = w[~counts].sum()
            m, w = m[counts], w[counts]
            p, va = w / w.sum(), np.abs(vv[m])
            e = 2 * D * 2.0 ** -24 * mag[i, m] + 2.0 ** -20 + (len(m) + 1) * 2.0 ** -24
            pv, top = p @ va, va.max()
            out[i, h] = p @ vv[m]
            b = (p * e) @ va + (p @ e) * pv + (2.0 ** -22 + 2 * len(m) * 2.0 ** -23 + 2.0 ** -20) * pv
            b += (len(m) * 2.0 ** -32 + 2 * lost) * top
            bound[i, h] = b * (1 + half) + half * np.abs(out[i, h]) + 2.0 ** -25
            first = (w * 128).astype(np.float16).astype(np.float64) / 128
            one[i, h] = first @ vv[m] / w.sum()
            off[i, h] = (first + np.roll(w - first, 1)) @ vv[m] / w.sum()
    return out, bound, one, off


# 64, 128 and 256 rows to an item; heads of 64 and 128; with one and several groups
@pytest.mark.parametrize("D,group,G,size", [(128, 128, 4, 16), (128, 32, 8, 5), (128, 64, 8, 14), (64, 64, 7, 9), (64, 32, 12, 10),
                                            (128, 128, 8, 18), (64, 32, 16, 9), (64, 64, 8, 33)])
@pytest.mark.parametrize("lse", [True, False])
@pytest.mark.parametrize("cut", [True, False])
def test_weights_enter_in_two_parts(D, group, G, size, lse, cut):
    if cut:
        c = prepared([6000, 2500, size + 9, 4001], [size, size, size, 3], 7, True, 1, G, D, group, seed=size)
    else:  # more blocks than the kernel for few rows takes
        c = prepared([size + int(x) for x in np.random.default_rng(size).integers(5, 190, 64)], [size] * 64, 5, False, 1, G, D, group, seed=D + size)
    rows = size * G
    assert cut or rows > 128 or -(-rows // 8) * 64 > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    out, _ = c.run(lse=lse)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    pool, r, told, moved, total = c.pool.cpu().numpy(), 0, 0, 0, 0
    for b, (T, n, base) in enumerate(zip(c.lens, c.new, c.base)):
        k, v, _, _ = ref.read_sequence(pool, c.table[b], T, c.Hkv, D, group, c.P)
        ok = tr.seen(T, base, c.masks[b], c.words, 0)
        want, bound, one, off = statement(c.q[r:r + n].double().cpu().numpy(), k, v, 1 / math.sqrt(D), ok)
        far = np.abs(out[r:r + n].double().cpu().numpy() - want)
        assert (far <= bound).all(), f"sequence {b}: {(far - bound).max():.3e} beyond the bound ({(far / bound).max():.2f} of it)"
        told += (np.abs(one - want) > bound).sum()
        moved += (np.abs(off - want) > bound).sum()
        total += want.size
        r += n
    assert told > total / 50 and moved > total / 50  # what the bound would not let pass


@pytest.mark.parametrize("D,group,G,size", [(128, 128, 8, 20), (128, 32, 8, 40), (64, 64, 7, 9), (64, 32, 16, 20), (64, 64, 8, 5), (128, 64, 8, 14)])
@pytest.mark.parametrize("wide", [True, False])
def test_fp16_outputs_do_not_go_by_the_log_sum_exp(D, group, G, size, wide):
    """Keys are exact whether it is asked for or not."""
    c = Tree([700 + size, 90 + size, size], [size, size, size], Hkv=2, G=G, D=D, group=group, P=16, dtype="fp16", seed=size)
    if wide:
        c.table = np.ascontiguousarray(np.concatenate([c.table, np.full((3, 2 ** 20 // c.P), 10 ** 6, np.int32)], 1))
    (a, _), (b, _) = c.run(lse=True), c.run(lse=False)
    torch.cuda.synchronize()
    assert int(c.err) == 0 and torch.equal(a, b)

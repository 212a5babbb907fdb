"""Verification of drafted tokens over rows as long as served vocabularies: parts of a warp of several rounds, new tokens looked for
in a warp's part by the whole CTA, few sequences and many; against whole numbers, so every result is equal."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import tree_ref as tr, verify_ref as vr
from tests.test_gpu_kv4 import error_word, ints, offsets
from tests.test_gpu_verify import rows_of, softmax32

pytestmark = pytest.mark.gpu
# a chain, siblings under the root and deeper, a root alone
SHAPES = [[-1, 0, 1, 2], [-1, 0, 0, 0], [-1, 0, 0, 1, 1], [-1], [-1, 0, 1, 1, 1]]


def strided(rows, shift, width):
    """The rows in a wider array, so that they begin at odd places."""
    wide = torch.full((len(rows), width), float("nan"), device="cuda")
    wide[:, shift:shift + rows.shape[1]] = torch.tensor(rows).cuda()
    return wide[:, shift:shift + rows.shape[1]]


def borders(rng, V, n):
    """Entries at which warps' parts, rounds and rows begin or end."""
    some = [0, 1, V - 1, V - 2] + [128 * int(rng.integers(0, V // 128 + 1)) + int(rng.integers(-4, 5)) for _ in range(n)]
    return [min(max(x, 0), V - 1) for x in some][:n]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,B,shift,pad", [(33000, 3, 0, 0), (65537, 3, 1, 6), (102401, 3, 3, 2), (150001, 3, 2, 1),  # 512 threads to a CTA
                                           (17000, 40, 1, 3), (40002, 40, 0, 2), (65537, 40, 2, 1)])                    # 256
def test_sampled_over_served_vocabularies(V, B, shift, pad, drawn):
    rng = np.random.default_rng(V + B + drawn)
    parents = [SHAPES[b % len(SHAPES)] for b in range(B)]
    sizes = [len(p) for p in parents]
    few = 5  # rows that differ; every sequence has rows among them
    z = rng.standard_normal((few, V))
    p, d = softmax32(z), softmax32(z + 0.7 * rng.standard_normal((few, V)))
    assign = lambda b, i: (b + 2 * i) % few  # noqa: E731
    of = np.array([assign(b, i) for b, n in enumerate(sizes) for i in range(n)])
    tokens, r = np.zeros(len(of), np.int64), 0
    for b, ps in enumerate(parents):
        for i, a in enumerate(ps):
            if a >= 0:
                row = d[assign(b, a)].astype(np.float64)
                tokens[r + i] = rng.choice(V, p=row / row.sum()) if drawn else np.argsort(-row)[(i + b) % 9]
        r += len(ps)
    # every third node of a sequence is accepted where anything of its token is left, the others are refused: none, one or several
    # before it (a picked child is accepted below its probability, ~1e-4 here)
    place = np.array([b + i for b, n in enumerate(sizes) for i in range(n)])
    ua = np.where(place % 3 == 1, rng.random(len(of)) * (0.3 if drawn else 0), 1 - 2.0 ** -24).astype(np.float32)
    P, Q = vr.Rows(p), vr.Rows(d) if drawn else None

    class Of:  # the sequence's rows by their place in the call
        def __init__(self, held):
            self.held, self.rows = held, held.rows

        def __getitem__(self, r):
            return self.held[of[r]]
    want, samplers, r = [], [], 0
    for b, ps in enumerate(parents):
        kept, new, rest = vr.walk(Of(P), None if Q is None else Of(Q), tokens[r:r + len(ps)], ps, ua[r:r + len(ps)], r)
        want.append((kept, new))
        samplers.append(vr.Sampler(rest))
        r += len(ps)
    assert len({tuple(k) for k, _ in want}) > 1
    target = strided(p[of], shift, V + 8 + pad)
    draft = strided(d[of], (3 * shift + 1) % 4 if pad else shift, V + 8 + pad) if drawn else None
    most = max(sizes)
    kept, new, count, err = ints(np.zeros((B, most))), ints(np.zeros((B, most))), ints([0] * B), error_word()
    mask, cu, tok = tr.mask_tensor([m for x in parents for m in tr.masks(x)], 1), offsets(sizes), ints(tokens)
    rounds = 24 if B < 10 else 4
    for k in range(rounds):
        at = borders(rng, V, B + k)[-B:] if k else [0, V - 1, V // 2] * B
        us = np.array([s.number_for(at[b]) for b, s in enumerate(samplers)], np.float32)
        q.mla_qcache_verify_sampled(target, tok, cu, most, torch.tensor(ua, device="cuda"), torch.tensor(us, device="cuda"), kept, new,
                                    count, err, draft_probs=draft, tree_mask=mask)
        torch.cuda.synchronize()
        assert int(err) == 0
        news = [w[1] + [s(u)] for w, s, u in zip(want, samplers, us)]
        assert count.tolist() == [len(w[0]) for w in want]
        assert np.array_equal(kept.cpu().numpy(), rows_of([w[0] for w in want], most))
        assert np.array_equal(new.cpu().numpy(), rows_of(news, most))


@pytest.mark.parametrize("V", [33001, 150001])
def test_picked_children_that_go_from_a_warps_part(V):
    """Many refused children whose entries lie side by side and far apart: they are gone from the sums and from the running sum."""
    rng = np.random.default_rng(V)
    n, B = 40, 2
    ps = [-1] + [0] * (n - 1)
    p = softmax32(rng.standard_normal((B, V)) * 0.3)
    tokens = np.concatenate([np.concatenate([[0], rng.integers(0, V, 9), 12800 + np.arange(15), [V - 1, V - 2, 0, 1, 2], rng.integers(0, V, 10)])
                             for _ in range(B)])
    ua = np.full(B * n, 1 - 2.0 ** -24, np.float32)
    samplers = [vr.Sampler(vr.walk(vr.Rows(p), None, tokens[b * n:], ps, ua, b)[2]) for b in range(B)]
    rows = torch.tensor(p).cuda().repeat_interleave(n, 0)
    kept, new, count, err = ints(np.zeros((B, n))), ints(np.zeros((B, n))), ints([0] * B), error_word()
    for at in [0, 3, 127, 128, 12799, 12805, 12815, 12900, V // 2, V - 3, V - 1] + [int(x) for x in rng.integers(0, V, 10)]:
        us = np.array([s.number_for(at) for s in samplers], np.float32)
        q.mla_qcache_verify_sampled(rows, ints(tokens), offsets([n] * B), n, torch.tensor(ua, device="cuda"), torch.tensor(us, device="cuda"),
                                    kept, new, count, err, tree_mask=tr.mask_tensor(tr.masks(ps) * B, 1))
        torch.cuda.synchronize()
        assert int(err) == 0 and count.tolist() == [1] * B
        assert new[:, 0].tolist() == [s(u) for s, u in zip(samplers, us)]


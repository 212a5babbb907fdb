"""Decoding with trees of drafted tokens as a server runs it: append the tree, attend, verify, keep, over several steps, against a
cache that the accepted tokens alone entered one after another."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import tree_ref as tr
from tests.test_gpu_kv4 import ints, offsets, tables

pytestmark = pytest.mark.gpu
VOCAB, HQ, HKV, D, P, B = 50, 8, 2, 128, 16, 3
SCALE = D ** -0.5


class Model:
    """One layer whose queries, keys and values go by the token alone, and a head on its attention's output."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.q, self.k, self.v = (rnd(VOCAB, h, D).bfloat16() for h in (HQ, HKV, HKV))
        self.head = rnd(HQ * D, VOCAB) * 0.3
        cos, sin = tables(512, D)
        self.cos, self.sin = torch.tensor(cos).cuda(), torch.tensor(sin).cuda()

    def rows(self, cache, tokens, cu, most, **kw):
        """Appends the tokens and attends: (output, logits)."""
        t = tokens.long()
        turned = torch.empty(len(t), HQ, D, dtype=torch.bfloat16, device="cuda")
        cache.append(self.k[t], self.v[t], cu, most, cos=self.cos, sin=self.sin, q=self.q[t], q_out=turned, **kw)
        out = cache.attend(turned, SCALE, cu_q=cu, max_q=most, **kw)
        return out, out.flatten(1).float() @ self.head


def prompt(model, seed):
    rng = np.random.default_rng(seed)
    cache = q.KV4Cache(q.make_kv4_config(HKV, D, page_size=P), B, 12)
    lens = [5, 37, 16]
    tokens = [rng.integers(0, VOCAB, n) for n in lens]
    model.rows(cache, ints(np.concatenate(tokens)), offsets(lens), max(lens))
    return cache, [list(t) for t in tokens], rng


def held(cache, n):
    """Bytes of the first n[b] tokens of each sequence."""
    pool, table = cache.pool.cpu().numpy(), cache.page_table.cpu().numpy()
    return [b"".join(x.tobytes() for t in range(k) for h in range(HKV) for x in tr.token_bytes(pool, table[b, t // P], t % P, h, D, D, P))
            for b, k in enumerate(n)]


@pytest.mark.parametrize("nodes,greedy", [(6, True), (6, False), (30, True), (30, False)])
def test_steps_leave_the_cache_as_if_the_accepted_tokens_had_come_one_by_one(nodes, greedy):
    model = Model(nodes)
    cache, text, rng = prompt(model, 1)
    plain, _, _ = prompt(model, 1)
    last = [int(x) for x in rng.integers(0, VOCAB, B)]
    kept, new, count, err = ints(np.zeros((B, nodes))), ints(np.zeros((B, nodes))), ints([0] * B), ints([0])
    accepted = 0
    for step in range(4):
        parents = [tr.random_parents(rng, nodes, 4) for _ in range(B)]
        tokens = rng.integers(0, VOCAB, (B, nodes))
        tokens[:, 0] = last
        cu = offsets([nodes] * B)
        mask = torch.empty(B * nodes, dtype=torch.int64, device="cuda")
        q.mla_qcache_tree_mask(ints([x for p in parents for x in p]), cu, nodes, mask, err)
        if greedy:  # a draft that is right most of the time: look at what the tree's rows will choose, level by level
            for _ in range(nodes):
                trial = q.KV4Cache(cache.cfg, B, 12, page_table=cache.page_table)
                trial.pool.copy_(cache.pool), trial.seq_lens.copy_(cache.seq_lens)
                trial.start_tree()
                best = model.rows(trial, ints(tokens.reshape(-1)), cu, nodes, tree_mask=mask)[1].argmax(1).view(B, nodes).cpu().numpy()
                fixed = tokens.copy()
                for b in range(B):
                    for i in range(1, nodes):
                        if i % 3:
                            fixed[b, i] = best[b, parents[b][i]]
                if (fixed == tokens).all():
                    break
                tokens = fixed
        cache.start_tree()
        before = cache.seq_lens.tolist()
        out, logits = model.rows(cache, ints(tokens.reshape(-1)), cu, nodes, tree_mask=mask)
        assert cache.seq_lens.tolist() == [x + nodes for x in before]
        if greedy:
            q.mla_qcache_verify_greedy(logits, ints(tokens.reshape(-1)), cu, nodes, kept, new, count, err, tree_mask=mask)
        else:
            p = torch.softmax(logits, -1)
            q.mla_qcache_verify_sampled(p, ints(tokens.reshape(-1)), cu, nodes, torch.rand(B * nodes, device="cuda") * 0.05,
                                        torch.rand(B, device="cuda"), kept, new, count, err, tree_mask=mask)
        cache.keep(kept, count)
        torch.cuda.synchronize()
        assert int(err) == 0 and cache.error_bits() == 0
        n = count.tolist()
        assert cache.seq_lens.tolist() == [x + y for x, y in zip(before, n)]
        # the same tokens one by one
        for i in range(max(n)):
            take = [i < x for x in n]
            cu1 = offsets([int(x) for x in take])
            t = [tokens[b, kept[b, i]] for b in range(B) if take[b]]
            o1, _ = model.rows(plain, ints(t), cu1, 1)
            # both are rounded to BF16 (2^-8 of them each), and their weights, and the values of the kernel for many rows, to FP16:
            # three roundings of 2^-11 of at most the largest value, on either side
            tol = 2 * 2.0 ** -8 * o1.float().abs() + 6 * 2.0 ** -11 * model.v.float().abs().max()
            o2 = out[[b * nodes + int(kept[b, i]) for b in range(B) if take[b]]]
            assert ((o1.float() - o2.float()).abs() <= tol).all()
        assert plain.seq_lens.tolist() == cache.seq_lens.tolist()
        assert held(cache, cache.seq_lens.tolist()) == held(plain, plain.seq_lens.tolist())
        last = [int(new[b, n[b] - 1]) for b in range(B)]
        accepted += sum(n) - B
    assert accepted > 0  # the path was taken at all


def test_a_captured_step_is_replayed():
    """One graph holds the whole step; its replays go on from the lengths that the one before left."""
    model, nodes = Model(3), 7
    eager, _, rng = prompt(model, 2)
    cache, _, _ = prompt(model, 2)
    parents = [tr.random_parents(rng, nodes, 4) for _ in range(B)]
    cu = offsets([nodes] * B)
    mask = tr.mask_tensor([m for p in parents for m in tr.masks(p)], 1)[:, 0].contiguous()
    tokens, ua, us = ints(np.zeros(B * nodes)), torch.zeros(B * nodes, device="cuda"), torch.zeros(B, device="cuda")

    def step(c, kept, new, count, err):
        c.start_tree()
        _, logits = model.rows(c, tokens, cu, nodes, tree_mask=mask)
        q.mla_qcache_verify_sampled(torch.softmax(logits, -1), tokens, cu, nodes, ua, us, kept, new, count, err, tree_mask=mask)
        c.keep(kept, count)
    state = [[ints(np.zeros((B, nodes))), ints(np.zeros((B, nodes))), ints([0] * B), ints([0])] for _ in range(2)]
    warm, _, _ = prompt(model, 2)
    step(warm, *state[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cache, *state[1])
    for _ in range(4):
        tokens.copy_(ints(rng.integers(0, VOCAB, B * nodes)))
        ua.copy_(torch.tensor(rng.random(B * nodes) * 0.1)), us.copy_(torch.tensor(rng.random(B)))
        step(eager, *state[0])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(*state)) and int(state[0][3]) == 0
        assert eager.seq_lens.tolist() == cache.seq_lens.tolist() and cache.error_bits() == 0
        n = cache.seq_lens.tolist()
        assert held(cache, n) == held(eager, n)

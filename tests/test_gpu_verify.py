"""Verification of drafted tokens on the GPU against the statement in rational numbers (tree_ref): whole numbers, so every result is
equal."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import tree_ref as tr
from tests.test_gpu_kv4 import error_word, ints, offsets

pytestmark = pytest.mark.gpu
F32 = torch.float32


def softmax32(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def call_sampled(target, draft, tokens, sizes, ua, us, ms=None, words=1, max_rows=None, stream=None):
    """target, draft: CUDA tensors (rows may be strided)."""
    B, most = len(sizes), max_rows or max(1, max(sizes))
    kept, new, n = ints(np.full((B, most), 77)), ints(np.full((B, most), 77)), ints([77] * B)
    err = error_word()
    q.mla_qcache_verify_sampled(target, ints(tokens), offsets(sizes), most, torch.tensor(ua, dtype=F32, device="cuda"),
                                torch.tensor(us, dtype=F32, device="cuda"), kept, new, n, err, draft_probs=draft,
                                tree_mask=None if ms is None else tr.mask_tensor(ms, words), stream=stream)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy(), n.tolist(), int(err)


def rows_of(lists, most):
    out = np.full((len(lists), most), -1, np.int64)
    for i, x in enumerate(lists):
        out[i, :len(x)] = x
    return out


def check_sampled(target, draft, tokens, parents, ua, us, got, most):
    kept, new, n, _ = got
    r, want = 0, []
    for b, ps in enumerate(parents):
        k = len(ps)
        cut = lambda x: None if x is None else x[r:r + k]  # noqa: E731
        want.append(tr.verify_sampled(cut(target), cut(draft), tokens[r:r + k], ps, ua[r:r + k], us[b]) if k else ([], []))
        r += k
    assert n == [len(w[0]) for w in want]
    assert np.array_equal(kept, rows_of([w[0] for w in want], most))
    assert np.array_equal(new, rows_of([w[1] for w in want], most))
    return want


def make(rng, sizes, V, chain, drawn, sharp=2.0, near=0.5):
    parents = [[i - 1 for i in range(n)] if chain else tr.random_parents(rng, n) if n else [] for n in sizes]
    rows = sum(sizes)
    z = rng.standard_normal((rows, V)) * sharp
    target = softmax32(z)
    draft = softmax32(z + near * rng.standard_normal((rows, V)))
    tokens, r = np.zeros(rows, np.int64), 0
    for ps in parents:
        used = {}
        for i, p in enumerate(ps):
            if p >= 0:
                d = draft[r + p].astype(np.float64)
                if drawn:
                    tokens[r + i] = rng.choice(V, p=d / d.sum())
                else:
                    tokens[r + i] = np.argsort(-d)[used.get(p, 0) % V]
                    used[p] = used.get(p, 0) + 1
        r += len(ps)
    ua = rng.random(rows).astype(np.float32)
    us = rng.random(len(sizes)).astype(np.float32)
    return parents, target, draft if drawn else None, tokens, ua, us


@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 31, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("drawn", [True, False])
def test_every_result_is_the_statements(V, chain, drawn):
    rng = np.random.default_rng(V + 10 * chain + 100 * drawn)
    sizes = [4, 1, 0, 6, 2, 9] if V < 1000 else [5, 3]
    ps, p, d, t, ua, us = make(rng, sizes, V, chain, drawn)
    cuda = lambda x: None if x is None else torch.tensor(x).cuda()  # noqa: E731
    ms = None if chain else [m for x in ps for m in (tr.masks(x) if x else [])]
    got = call_sampled(cuda(p), cuda(d), t, sizes, ua, us, ms)
    assert got[3] == 0
    check_sampled(p, d, t, ps, ua, us, got, max(sizes))


def test_many_small_cases():
    """Hundreds of trees with few tokens, so that every branch is taken: equal siblings, rejections of all, bonus tokens."""
    for seed, (V, drawn) in enumerate([(4, True), (4, False), (9, True), (9, False), (40, True)]):
        rng = np.random.default_rng(seed)
        sizes = [int(x) for x in rng.integers(1, 13, 120)]
        ps, p, d, t, ua, us = make(rng, sizes, V, False, drawn, sharp=1.0, near=1.5)
        got = call_sampled(torch.tensor(p).cuda(), None if d is None else torch.tensor(d).cuda(), t, sizes, ua, us,
                           [m for x in ps for m in tr.masks(x)], words=4)
        want = check_sampled(p, d, t, ps, ua, us, got, max(sizes))
        assert got[3] == 0 and len({len(w[0]) for w in want}) > 2


@pytest.mark.parametrize("drawn", [True, False])
def test_sums_that_are_exact_borders(drawn):
    """Probabilities and random numbers that are multiples of 1/64: the running sum meets u times the whole exactly, and a token
    is accepted only below the border."""
    V, B = 64, 64
    p = np.full((2 * B, V), 1 / 64, np.float32)
    d = p.copy()
    if drawn:  # the draft is sure of half of the tokens
        d[:] = 0
        d[:, :32] = 1 / 32
    t = np.tile([0, 5], B)
    ua = np.repeat(np.arange(B) / 64, 2).astype(np.float32)  # accepted while u < 1/2 (drawn), u < 1/64 (picked)
    us = (np.arange(B) / 64).astype(np.float32)
    got = call_sampled(torch.tensor(p).cuda(), torch.tensor(d).cuda() if drawn else None, t, [2] * B, ua, us)
    check_sampled(p, d if drawn else None, t, [[-1, 0]] * B, ua, us, got, 2)
    assert got[2] == [2 if u < (0.5 if drawn else 1 / 64) else 1 for u in ua[::2]]


def test_numbers_that_do_not_count():
    """Negative, infinite and NaN entries count as 0; a row without any gives -1 and is reported; random numbers of 1 or NaN stay in
    range; tokens outside the vocabulary are never accepted."""
    V = 300
    rng = np.random.default_rng(0)
    p = softmax32(rng.standard_normal((7, V)))
    p[0, :100], p[1, 7], p[1, 8], p[1, 9] = np.nan, np.inf, -np.inf, -0.5
    p[2] = 0
    p[3] = np.nan
    p[4, 1:] = 0
    d = softmax32(rng.standard_normal((7, V)))
    d[0, 5], d[1, 20] = np.nan, np.inf
    t = np.array([0, 250, 0, -1, 0, V, 2 ** 31 - 1])
    sizes = [2, 1, 1, 1, 2]
    for draft in (d, None):
        for us in (0.0, 0.3, np.float32(1 - 2.0 ** -24)):
            ua, u = np.full(7, 0.999, np.float32), np.full(5, us, np.float32)
            got = call_sampled(torch.tensor(p).cuda(), None if draft is None else torch.tensor(draft).cuda(), t, sizes, ua, u)
            assert got[3] == q.DEV_RANGE
            check_sampled(p, draft, t, [[-1, 0], [-1], [-1], [-1], [-1, 0]], ua, u, got, 2)
    for us in (1.0, 5.0, float("nan"), float("inf"), -1.0):
        got = call_sampled(torch.tensor(p[4:]).cuda(), torch.tensor(d[4:]).cuda(), [0, 0, 0], [1, 1, 1], [np.nan] * 3, [us] * 3)
        assert got[2] == [1, 1, 1] and got[1][0, 0] == 0 and all(0 <= x < V for x in got[1][:, 0])
    assert call_sampled(torch.tensor(p[5:]).cuda(), torch.tensor(d[5:]).cuda(), [0, 3], [2], [0, np.nan], [0.5])[2] == [1]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,at", [(50, 0), (100000, 0), (100000, 60000), (100000, 99990)])
def test_a_sum_that_overflows_gives_no_token(V, at, drawn):
    """Wherever in the row it overflows, and whatever else the row holds; the sequences beside it are answered."""
    big = float(np.finfo(np.float32).max)
    p = torch.full((4, V), 1 / V, device="cuda")
    p[1, at:at + 3] = big
    d = torch.full((4, V), 1 / V, device="cuda") if drawn else None
    got = call_sampled(p, d, [0, -1, -1, -1], [1, 2, 1], [0.5] * 4, [0.5] * 3)
    assert got[3] == q.DEV_RANGE and got[2] == [1, 1, 1]
    assert got[1][1, 0] == -1 and abs(got[1][0, 0] - V // 2) <= 1 and abs(got[1][2, 0] - V // 2) <= 1


@pytest.mark.parametrize("drawn", [True, False])
def test_equal_distributions_accept_and_leave_nothing(drawn):
    """p = q: a draft is accepted whatever the number; one with p(x) = q(x) = 0 is refused, nothing is left, and p is drawn from."""
    V = 50
    p = softmax32(np.random.default_rng(1).standard_normal((6, V)))
    p[:, 9] = 0
    t = np.array([0, 3, 9, 0, 9, 9])
    ps = [[-1, 0, 1], [-1, 0, 0]]
    ua, us = np.full(6, np.float32(1 - 2.0 ** -24)), np.array([0.2, 0.8], np.float32)
    d = p if drawn else None
    got = call_sampled(torch.tensor(p).cuda(), torch.tensor(p).cuda() if drawn else None, t, [3, 3], ua, us,
                       [m for x in ps for m in tr.masks(x)])
    check_sampled(p, d, t, ps, ua, us, got, 3)
    assert got[3] == 0 and got[2][1] == 1


@pytest.mark.parametrize("V,shift", [(1000, 0), (1000, 1), (1003, 0), (1001, 3), (50, 2)])
def test_rows_of_any_alignment_and_stride(V, shift):
    rng = np.random.default_rng(V + shift)
    sizes = [4, 3]
    ps, p, d, t, ua, us = make(rng, sizes, V, True, True)
    wide_p, wide_d = torch.full((7, V + 9), float("nan"), device="cuda"), torch.full((7, 2 * V + 1), float("nan"), device="cuda")
    wide_p[:, shift:shift + V], wide_d[:, 1:1 + V] = torch.tensor(p).cuda(), torch.tensor(d).cuda()
    got = call_sampled(wide_p[:, shift:shift + V], wide_d[:, 1:1 + V], t, sizes, ua, us)
    check_sampled(p, d, t, ps, ua, us, got, 4)
    one = torch.tensor(p[:1]).cuda().expand(7, V)  # the same row for all
    got = call_sampled(one, torch.tensor(d).cuda(), t, sizes, ua, us)
    check_sampled(np.tile(p[:1], (7, 1)), d, t, ps, ua, us, got, 4)


def test_large_trees_and_padding():
    rng = np.random.default_rng(3)
    sizes = [256, 200, 65, 1]
    ps, p, d, t, ua, us = make(rng, sizes, 24, False, True, sharp=0.5, near=0.2)
    t[::7] = -1  # padded nodes
    got = call_sampled(torch.tensor(p).cuda(), torch.tensor(d).cuda(), t, sizes, ua, us, [m for x in ps for m in tr.masks(x)], words=4)
    check_sampled(p, d, t, ps, ua, us, got, 256)
    wide = [[-1] + [0] * 255]  # a root with 255 children
    p1, d1 = p[:256], d[:256]
    t1 = rng.integers(0, 24, 256)
    for draft in (d1, None):
        got = call_sampled(torch.tensor(p1).cuda(), None if draft is None else torch.tensor(draft).cuda(), t1, [256],
                           np.full(256, 0.99999, np.float32), [0.5], [m for m in tr.masks(wide[0])], words=4)
        check_sampled(p1, draft, t1, wide, np.full(256, 0.99999, np.float32), [0.5], got, 256)


@pytest.mark.parametrize("children", [1, 3])
def test_what_comes_out_is_the_targets_distribution(children):
    """40000 steps with the same p and q: the first token's frequencies are p's within five standard deviations."""
    V, B = 6, 40000
    rng = np.random.default_rng(children)
    p, d = softmax32(rng.standard_normal((1, V))), softmax32(rng.standard_normal((1, V)) * 1.5)
    n = children + 1
    t = rng.choice(V, size=(B, n), p=d[0].astype(np.float64) / d[0].astype(np.float64).sum()).reshape(-1)
    rows = lambda x: torch.tensor(x).cuda().expand(B * n, V)  # noqa: E731
    got = call_sampled(rows(p), rows(d), t, [n] * B, rng.random(B * n).astype(np.float32), rng.random(B).astype(np.float32),
                       tr.masks([-1] + [0] * children) * B)
    share = np.bincount(got[1][:, 0], minlength=V) / B
    assert (np.abs(share - p[0]) <= 5 * np.sqrt(p[0] * (1 - p[0]) / B)).all(), (share, p)


def test_sequences_that_do_not_fit_are_reported():
    rng = np.random.default_rng(9)
    ps, p, d, t, ua, us = make(rng, [3, 4, 2], 20, True, True)
    pc, dc = torch.tensor(p).cuda(), torch.tensor(d).cuda()
    kept, new, n, err = call_sampled(pc, dc, t, [3, 4, 2], ua, us, max_rows=3)
    assert err == q.DEV_ROWS and n[1] == 0 and (kept[1] == -1).all() and (new[1] == -1).all()
    check_sampled(p[:3], d[:3], t[:3], ps[:1], ua[:3], us[:1], (kept[:1], new[:1], n[:1], 0), 3)
    check_sampled(p[7:], d[7:], t[7:], ps[2:], ua[7:], us[2:], (kept[2:], new[2:], n[2:], 0), 3)


# ---------------------------------------------------------------- greedy
def call_greedy(logits, tokens, sizes, ms=None, words=1, max_rows=None):
    B, most = len(sizes), max_rows or max(1, max(sizes))
    kept, new, n, err = ints(np.full((B, most), 77)), ints(np.full((B, most), 77)), ints([77] * B), error_word()
    q.mla_qcache_verify_greedy(logits, ints(tokens), offsets(sizes), most, kept, new, n, err,
                               tree_mask=None if ms is None else tr.mask_tensor(ms, words))
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy(), n.tolist(), int(err)


def check_greedy(logits, tokens, parents, got):
    x, r, want = logits.double().cpu().numpy(), 0, []
    for ps in parents:
        want.append(tr.verify_greedy(x[r:r + len(ps)], tokens[r:r + len(ps)], ps) if ps else ([], []))
        r += len(ps)
    most = got[0].shape[1]
    assert got[2] == [len(w[0]) for w in want]
    assert np.array_equal(got[0], rows_of([w[0] for w in want], most)) and np.array_equal(got[1], rows_of([w[1] for w in want], most))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 1000, 4099, 40001])
def test_greedy_takes_the_first_of_the_largest(dtype, V):
    rng = np.random.default_rng(V)
    sizes = [5, 1, 0, 12, 3]
    ps = [tr.random_parents(rng, n) if n else [] for n in sizes]
    x = torch.tensor(np.round(rng.standard_normal((sum(sizes), V)) * 2) / 2, dtype=F32).to(dtype).cuda()  # many equal ones
    best = x.double().cpu().numpy().argmax(1)
    t, r = np.zeros(sum(sizes), np.int64), 0
    for p in ps:
        for i, a in enumerate(p):
            t[r + i] = best[r + a] if a >= 0 and rng.random() < 0.7 else int(rng.integers(-1, V + 1))
        r += len(p)
    got = call_greedy(x, t, sizes, [m for p in ps for m in (tr.masks(p) if p else [])])
    assert got[3] == 0
    check_greedy(x, t, ps, got)
    wide = torch.full((sum(sizes), V + 5), float("inf"), dtype=dtype, device="cuda")
    wide[:, 3:3 + V] = x
    chain = [list(range(-1, n - 1)) for n in sizes]
    check_greedy(x, t, chain, call_greedy(wide[:, 3:3 + V], t, sizes))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_greedy_over_infinities_zeros_and_no_numbers(dtype):
    V = 777
    x = torch.full((6, V), -float("inf"), dtype=dtype, device="cuda")
    x[0, 100:] = float("nan")                      # -inf and NaN: token 0
    x[1] = float("nan")                            # nothing: -1
    x[2, 5], x[2, 9] = float("inf"), float("inf")
    x[3, 7], x[3, 8], x[3, 6] = -0.0, 0.0, -1.0    # equal zeros: the first
    x[4, :50] = float("nan")
    x[4, 60] = -3.0
    got = call_greedy(x, [0] * 6, [1] * 6)
    assert got[1][:, 0].tolist() == [0, -1, 5, 7, 60, 0] and got[3] == q.DEV_NONFINITE and got[2] == [1] * 6
    # a row without a number ends the path, whatever its children carry
    got = call_greedy(x[1:3], [0, -1], [2])
    assert got[2] == [1] and got[1][0].tolist() == [-1, -1]


def test_greedy_of_large_trees():
    rng = np.random.default_rng(2)
    n, V = 256, 64
    x = torch.tensor(rng.standard_normal((n, V)), dtype=F32).cuda()
    best = x.cpu().numpy().argmax(1)
    chain = list(range(-1, n - 1))
    t = np.concatenate([[0], best[:-1]])  # all of a chain of 256 is right
    check_greedy(x, t, [chain], call_greedy(x, t, [n]))
    ps = tr.random_parents(rng, n, 3)
    t = np.array([0 if p < 0 else best[p] for p in ps])
    check_greedy(x, t, [ps], call_greedy(x, t, [n], tr.masks(ps), words=4))


def test_captured_calls_and_streams():
    rng = np.random.default_rng(4)
    sizes = [6] * 5
    ps, p, d, t, ua, us = make(rng, sizes, 500, True, True)
    pc, dc, tok = torch.tensor(p).cuda(), torch.tensor(d).cuda(), ints(t)
    uac, usc, cu = torch.tensor(ua).cuda(), torch.tensor(us).cuda(), offsets(sizes)
    kept, new, n, err = ints(np.zeros((5, 6))), ints(np.zeros((5, 6))), ints([0] * 5), error_word()
    call = lambda stream=None: q.mla_qcache_verify_sampled(pc, tok, cu, 6, uac, usc, kept, new, n, err, draft_probs=dc, stream=stream)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        _, p, d, t, ua, us = make(rng, sizes, 500, True, True)
        for to, x in ((pc, p), (dc, d), (uac, ua), (usc, us)):
            to.copy_(torch.tensor(x))
        tok.copy_(ints(t))
        g.replay()
        torch.cuda.synchronize()
        check_sampled(p, d, t, ps, ua, us, (kept.cpu().numpy(), new.cpu().numpy(), n.tolist(), 0), 6)
    s = torch.cuda.Stream()
    kept.fill_(5)
    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    check_sampled(p, d, t, ps, ua, us, (kept.cpu().numpy(), new.cpu().numpy(), n.tolist(), 0), 6)

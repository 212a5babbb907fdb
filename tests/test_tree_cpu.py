"""Trees of drafted tokens without a GPU: the plain statements against one another, and what the C ABI and the binding refuse before
any launch."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from bit_mla_kv_qcache_gb300 import binding
from tests import tree_ref as tr
from tests.test_kv4_cpu import P16, PFAR, _rot, _view, lib  # noqa: F401

ODD = ctypes.c_void_p(16 * 1024 + 2)
PB, PC = ctypes.c_void_p(1 << 41), ctypes.c_void_p(1 << 42)


def test_masks_and_parents_are_one_another():
    rng = np.random.default_rng(0)
    for n in (1, 2, 30, 64, 65, 256):
        p = tr.random_parents(rng, n)
        ms = tr.masks(p)
        assert tr.parents_of(ms) == p
        words = -(-n // 64)
        t = tr.mask_tensor(ms, words, "cpu")
        back = [sum((int(x) & (1 << 64) - 1) << 64 * w for w, x in enumerate(row)) for row in t]
        assert back == ms


def test_a_chains_mask_is_causal():
    ms = tr.masks(list(range(-1, 6)))
    assert (tr.seen(12, 5, ms, 1, 0) == (np.arange(12)[None] <= np.arange(5, 12)[:, None])).all()
    # a window covers the tokens before the tree by the node's depth
    assert [int(r[:5].sum()) for r in tr.seen(12, 5, ms, 1, 4)] == [3, 2, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("children", [1, 2, 3])
def test_the_statement_of_verification_gives_the_targets_distribution(children):
    """Exactly, by summing over the draws of the children and integrating over the random numbers: each branch's share is its
    bounds' length."""
    V = 3
    p = [Fraction(1, 2), Fraction(1, 8), Fraction(3, 8)]
    d = [Fraction(1, 4), Fraction(1, 2), Fraction(1, 4)]
    out = [Fraction(0)] * V

    def go(k, c, Z, share):
        left = [max(x - c * y, 0) for x, y in zip(p, d)]
        if k == children:
            total = sum(left)
            for j in range(V):
                out[j] += share * left[j] / total
            return
        for x in range(V):  # this child's token
            accept = min(Fraction(1), left[x] / (d[x] * Z))
            out[x] += share * d[x] * accept
            if accept < 1:
                c2 = c + Z
                go(k + 1, c2, sum(max(a - c2 * b, 0) for a, b in zip(p, d)), share * d[x] * (1 - accept))
    go(0, Fraction(0), Fraction(1), Fraction(1))
    assert out == p


def _tree(mask=P16, words=1, base=None):
    return ctypes.byref(binding._Tree(mask.value if mask else None, words, base.value if base else None))


def _attn_tree(lib, cfg=None, dtype=0, B=2, heads=8, rows=2, qv=..., cu=P16, max_q=1, tree=..., table=P16, pages=4, lens=P16,  # noqa: F811
               pool=P16, n_pages=4, window=0, scale=0.1, out=PFAR, lse=None, ws=P16, nbytes=1 << 40, err=P16):
    cfg = cfg or q.make_kv4_config(4)
    return lib.mla_qcache_kv4_attn_tree(ctypes.byref(cfg), dtype, B, heads, rows, _view() if qv is ... else qv, cu, max_q,
                                        _tree() if tree is ... else tree, table, pages, lens, pool, n_pages, window,
                                        ctypes.c_float(scale), out, lse, ws, nbytes, err, None)


def test_attention_refusals(lib):  # noqa: F811
    assert _attn_tree(lib, rows=0) == 0
    assert _attn_tree(lib, dtype=7) == -2 and _attn_tree(lib, cfg=q.make_kv4_config(4, 128, group=100)) == -2
    for kw in [dict(B=0), dict(heads=6), dict(rows=-1), dict(max_q=0), dict(max_q=65), dict(max_q=257, tree=_tree(words=4)),
               dict(tree=_tree(words=0)), dict(tree=_tree(words=5)), dict(tree=_tree(words=-1)), dict(tree=_tree(words=1 << 26)),
               dict(window=-1), dict(scale=float("nan")), dict(out=P16), dict(cu=None, rows=3)]:
        assert _attn_tree(lib, **kw) == -3, kw
    for kw in [dict(tree=None), dict(tree=_tree(None)), dict(qv=None), dict(table=None), dict(lens=None), dict(pool=None),
               dict(out=None), dict(ws=None), dict(err=None)]:
        assert _attn_tree(lib, **kw) == -1, kw
    for kw in [dict(tree=_tree(ctypes.c_void_p(16 * 1024 + 4))), dict(tree=_tree(base=ODD)), dict(out=ODD), dict(cu=ODD)]:
        assert _attn_tree(lib, **kw) == -4, kw


def _append_tree(lib, cfg=None, rows=2, tree=..., pool=PFAR, rot=None, kd=None, next=None):  # noqa: F811
    cfg = cfg or q.make_kv4_config(4)
    return lib.mla_qcache_kv4_append_tree(ctypes.byref(cfg), 0, 2, rows, _view(), _view(), P16, P16, next, 1, rot, None, 0, None, kd, None,
                                          P16, 4, pool, 4, _tree() if tree is ... else tree, P16, None)


def test_append_refusals(lib):  # noqa: F811
    assert _append_tree(lib, rows=0) == 0
    assert _append_tree(lib, tree=None) == -1 and _append_tree(lib, tree=_tree(None)) == -1
    for words in (0, 5, -3):
        assert _append_tree(lib, tree=_tree(words=words)) == -3
    assert _append_tree(lib, tree=_tree(ODD)) == -4 and _append_tree(lib, tree=_tree(base=ODD)) == -4
    assert _append_tree(lib, rot=_rot(dim=24)) == -3 and _append_tree(lib, kd=P16) == -3  # as the plain append


def test_outputs_over_masks_and_bases_are_refused(lib):  # noqa: F811
    near = ctypes.c_void_p(PFAR.value + 16)  # the second row's mask; base of the later sequences
    for tree in (_tree(PB, base=PFAR), _tree(PFAR, words=2), _tree(ctypes.c_void_p(PFAR.value - 24), words=2), _tree(PB, base=near)):
        assert _attn_tree(lib, tree=tree) == -3 and _append_tree(lib, tree=tree) == -3
    for tree in (_tree(PB), _tree(PC, base=PB)):
        assert _attn_tree(lib, tree=tree, lse=PB) == -3
        assert _append_tree(lib, tree=tree, next=PB) == -3
        assert _append_tree(lib, tree=tree, kd=PB) == -3


def _sampled(lib, B=2, rows=6, V=100, target=PFAR, ts=100, draft=PB, ds=100, tokens=P16, cu=P16, max_rows=3, mask=None, words=0,  # noqa: F811
             ua=P16, us=P16, kept=PC, new=ctypes.c_void_p((1 << 42) + 4096), n=ctypes.c_void_p((1 << 42) + 8192), err=P16):
    return lib.mla_qcache_verify_sampled(B, rows, V, target, ts, draft, ds, tokens, cu, max_rows, mask, words, ua, us, kept, new, n, err,
                                         None)


def _greedy(lib, dtype=0, B=2, rows=6, V=100, x=PFAR, stride=100, tokens=P16, cu=P16, max_rows=3, mask=None, words=0, kept=PC,  # noqa: F811
            new=ctypes.c_void_p((1 << 42) + 4096), n=ctypes.c_void_p((1 << 42) + 8192), err=P16):
    return lib.mla_qcache_verify_greedy(B, rows, V, dtype, x, stride, tokens, cu, max_rows, mask, words, kept, new, n, err, None)


def test_verification_refusals(lib):  # noqa: F811
    for call in (_sampled, _greedy):
        for kw in [dict(B=0), dict(B=(1 << 20) + 1), dict(rows=-1), dict(V=0), dict(max_rows=0), dict(max_rows=257),
                   dict(mask=P16, words=0), dict(mask=P16, words=5), dict(mask=P16, words=1, max_rows=65), dict(kept=P16),
                   dict(new=PC), dict(n=PC), dict(kept=PFAR)]:
            assert call(lib, **kw) == -3, (call, kw)
        for kw in [dict(tokens=None), dict(cu=None), dict(kept=None), dict(new=None), dict(n=None), dict(err=None)]:
            assert call(lib, **kw) == -1, (call, kw)
        for kw in [dict(tokens=ODD), dict(cu=ODD), dict(kept=ODD), dict(mask=ctypes.c_void_p(16 * 1024 + 4), words=1), dict(err=ODD)]:
            assert call(lib, **kw) == -4, (call, kw)
    for kw in [dict(ts=-1), dict(ds=-1), dict(ts=1 << 60), dict(ds=1 << 60), dict(kept=PB)]:
        assert _sampled(lib, **kw) == -3, kw
    assert _sampled(lib, target=None) == -1 and _sampled(lib, ua=None) == -1 and _sampled(lib, us=None) == -1
    assert _sampled(lib, target=ODD) == -4 and _sampled(lib, draft=ODD) == -4 and _sampled(lib, ua=ODD) == -4
    assert _greedy(lib, dtype=3) == -2 and _greedy(lib, dtype=-1) == -2
    assert _greedy(lib, x=None) == -1 and _greedy(lib, stride=-1) == -3
    assert _greedy(lib, x=ctypes.c_void_p(16 * 1024 + 1)) == -4 and _greedy(lib, dtype=2, x=ODD) == -4


def test_keep_and_mask_refusals(lib):  # noqa: F811
    cfg = q.make_kv4_config(2, page_size=16)

    def keep(c=cfg, B=2, kept=P16, most=8, n=P16, base=P16, table=P16, pages=4, pool=PFAR, n_pages=8, lens=PB, err=P16):
        return lib.mla_qcache_kv4_keep(ctypes.byref(c), B, kept, most, n, base, table, pages, pool, n_pages, lens, err, None)
    assert keep(c=q.make_kv4_config(0)) == -2
    for kw in [dict(B=0), dict(B=(1 << 20) + 1), dict(most=0), dict(most=257), dict(pages=0), dict(n_pages=0), dict(pages=1 << 28),
               dict(lens=P16), dict(pool=P16), dict(lens=PFAR), dict(base=PB), dict(table=PFAR)]:
        assert keep(**kw) == -3, kw
    for kw in [dict(kept=None), dict(n=None), dict(base=None), dict(table=None), dict(pool=None), dict(lens=None), dict(err=None)]:
        assert keep(**kw) == -1, kw
    for kw in [dict(kept=ODD), dict(base=ODD), dict(pool=ctypes.c_void_p((1 << 40) + 8)), dict(lens=ODD)]:
        assert keep(**kw) == -4, kw

    def mask(B=2, rows=4, parents=P16, cu=P16, most=8, words=1, out=PFAR, err=P16):
        return lib.mla_qcache_tree_mask(B, rows, parents, cu, most, words, out, err, None)
    assert mask(rows=0) == 0
    for kw in [dict(B=0), dict(rows=-1), dict(words=0), dict(words=5), dict(most=65), dict(most=0), dict(out=P16)]:
        assert mask(**kw) == -3, kw
    for kw in [dict(parents=None), dict(cu=None), dict(out=None), dict(err=None)]:
        assert mask(**kw) == -1, kw
    assert mask(out=ctypes.c_void_p((1 << 40) + 4)) == -4 and mask(parents=ODD) == -4


def test_binding_refuses_host_tensors(lib):  # noqa: F811
    cfg = q.make_kv4_config(8)
    z, i = torch.zeros(1, 8, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    ii, m, f = i.view(1, 1), torch.zeros(1, dtype=torch.int64), torch.zeros(1, 4)
    calls = [lambda: q.mla_qcache_kv4_attn_tree(cfg, z, m, i, 1, ii, i, z, 1.0, z, z, i),
             lambda: q.mla_qcache_kv4_append(cfg, z, z, i, i, 1, ii, z, i, tree_mask=m),
             lambda: q.mla_qcache_verify_sampled(f, i, i, 1, f, f, ii, ii, i, i),
             lambda: q.mla_qcache_verify_greedy(f, i, i, 1, ii, ii, i, i),
             lambda: q.mla_qcache_kv4_keep(cfg, ii, i, i, ii, z, i, i),
             lambda: q.mla_qcache_tree_mask(i, i, 1, m, i)]
    for c in calls:
        with pytest.raises(q.QCacheError, match="CUDA"):
            c()
    with pytest.raises(q.QCacheError, match="required"):
        q.mla_qcache_verify_greedy(None, i, i, 1, ii, ii, i, i)
    with pytest.raises(TypeError):
        q.mla_qcache_kv4_keep(cfg, 3, i, i, ii, z, i, i)

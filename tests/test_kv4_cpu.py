"""Grouped-query cache in 4 bits and the BF16 append without a GPU: the layout formulas are permutations,
the quantizer's plain statement holds its bounds, the C ABI refuses bad calls before any launch, and the
binding refuses tensors that it cannot pass on."""
import ctypes

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from bit_mla_kv_qcache_gb300 import binding
from tests import kv4_ref as ref

P16 = ctypes.c_void_p(16 * 1024)  # never dereferenced: every call below is refused first
PFAR = ctypes.c_void_p(1 << 40)


@pytest.fixture(scope="module")
def lib():
    from bit_mla_kv_qcache_gb300 import build
    build.build()
    return q.lib()


@pytest.mark.parametrize("D", [64, 128])
def test_channel_orders_are_permutations(D):
    assert sorted(ref.key_nibble(c, D) for c in range(D)) == list(range(D))
    assert sorted(ref.value_nibble(c, D) for c in range(D)) == list(range(D))
    codes = np.random.default_rng(0).integers(0, 16, (3, D)).astype(np.uint8)
    for nib in (ref.key_nibble, ref.value_nibble):
        assert np.array_equal(ref.unpack_rows(ref.pack_rows(codes, nib, D), nib, D), codes)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantizer_statement_is_within_half_a_scale(group):
    x = np.random.default_rng(group).standard_normal((50, 128)).astype(np.float32).astype(np.float64)
    x[0] = 3.25          # a constant group: scale 0, the minimum holds it
    x[1] = 0.0
    x[2, ::2], x[2, 1::2] = -1e-7, 1e-7  # FP16 subnormals
    n, s, m = ref.quantize(x, group)
    err = np.abs(ref.values(n, s, m, group) - x).reshape(50, -1, group)
    assert (err <= s.astype(np.float64)[..., None] / 2).all()
    assert (s[0] == 0).all() and (n[0] == 0).all() and (m[0] == 3.25).all()


def test_config_and_page_bytes(lib):
    assert q.kv4_page_bytes(q.make_kv4_config(8, 128, page_size=64)) == 8 * 64 * 136
    assert q.kv4_page_bytes(q.make_kv4_config(2, 64, group=32, page_size=16)) == 2 * 16 * 80
    bad = [q.make_kv4_config(0), q.make_kv4_config(257), q.make_kv4_config(1, 96), q.make_kv4_config(1, 64, group=128),
           q.make_kv4_config(1, 128, group=16), q.make_kv4_config(1, 128, page_size=48), q.make_kv4_config(1, 128, page_size=8)]
    for c in bad:
        assert lib.mla_qcache_kv4_config_check(ctypes.byref(c)) == -2
        assert q.kv4_page_bytes(c) == 0
        assert q.kv4_workspace_bytes(c, 1, 8, 1, 1) == 0
    assert lib.mla_qcache_kv4_config_check(None) == -1
    good = q.make_kv4_config(4)
    for args in [(0, 8, 1, 1), (1, 6, 1, 1), (1, 8, 0, 1), (1, 8, 1, 0), (1, 4097 * 4, 1, 1)]:
        assert q.kv4_workspace_bytes(good, *args) == 0


def _view(p=P16, row=512, head=128):
    return ctypes.byref(binding._View(p.value if p else None, row, head))


def _rot(p=P16, n_pos=8, dim=128):
    return ctypes.byref(binding._Rotation(p.value if p else None, p.value if p else None, n_pos, dim, 0))


def _append(lib, cfg=None, dtype=0, B=2, rows=2, k=..., v=..., cu=P16, lens=P16, nxt=None, max_new=1, rot=None, qv=None, heads=0,
            q_out=None, kd=None, vd=None, table=P16, pages=4, pool=PFAR, n_pages=4, err=P16):
    cfg = cfg or q.make_kv4_config(4)
    return lib.mla_qcache_kv4_append(ctypes.byref(cfg), dtype, B, rows, _view() if k is ... else k, _view() if v is ... else v, cu,
                                     lens, nxt, max_new, rot, qv, heads, q_out, kd, vd, table, pages, pool, n_pages, err, None)


def test_append_refusals(lib):
    assert _append(lib, rows=0) == 0  # nothing to do
    assert _append(lib, cfg=q.make_kv4_config(4, 96)) == -2
    assert _append(lib, dtype=2) == -2
    for kw in [dict(B=0), dict(B=(1 << 20) + 1), dict(rows=-1), dict(max_new=0), dict(pages=0), dict(n_pages=0),
               dict(k=_view(row=-512)), dict(rot=_rot(dim=24)), dict(rot=_rot(dim=144)), dict(rot=_rot(dim=0)),
               dict(rot=_rot(n_pos=0)), dict(qv=_view(), heads=0, q_out=PFAR), dict(qv=_view(), heads=5000, q_out=PFAR)]:
        assert _append(lib, **kw) == -3, kw
    for kw in [dict(k=None), dict(v=None), dict(k=_view(None)), dict(cu=None), dict(lens=None), dict(table=None),
               dict(pool=None), dict(err=None), dict(qv=_view(), heads=8), dict(q_out=PFAR), dict(rot=_rot(None))]:
        assert _append(lib, **kw) == -1, kw
    odd = ctypes.c_void_p(16 * 1024 + 8)
    two = ctypes.c_void_p(16 * 1024 + 2)
    for kw in [dict(k=_view(odd)), dict(k=_view(row=516)), dict(v=_view(head=4)), dict(pool=odd), dict(kd=odd), dict(cu=two),
               dict(err=two), dict(rot=_rot(odd))]:
        assert _append(lib, **kw) == -4, kw
    # outputs over inputs or over one another; the two length arrays over each other
    assert _append(lib, kd=P16) == -3
    assert _append(lib, kd=PFAR, vd=ctypes.c_void_p((1 << 41)), pool=ctypes.c_void_p(1 << 40)) == -3
    assert _append(lib, qv=_view(PFAR), heads=8, q_out=PFAR, pool=ctypes.c_void_p(1 << 42)) == -3
    assert _append(lib, nxt=ctypes.c_void_p(16 * 1024 + 4)) == -3


def _attn(lib, cfg=None, dtype=0, B=2, heads=8, rows=2, qv=..., cu=None, max_q=1, table=P16, pages=4, lens=P16, pool=P16, n_pages=4,
          causal=1, window=0, scale=0.1, out=PFAR, lse=None, ws=P16, nbytes=1 << 40, err=P16):
    cfg = cfg or q.make_kv4_config(4)
    return lib.mla_qcache_kv4_attn(ctypes.byref(cfg), dtype, B, heads, rows, _view() if qv is ... else qv, cu, max_q, table, pages,
                                   lens, pool, n_pages, causal, window, ctypes.c_float(scale), out, lse, ws, nbytes, err, None)


def test_attention_refusals(lib):
    assert _attn(lib, rows=0, cu=P16) == 0
    assert _attn(lib, dtype=7) == -2 and _attn(lib, cfg=q.make_kv4_config(4, 128, group=100)) == -2
    for kw in [dict(B=0), dict(heads=0), dict(heads=6), dict(heads=4100), dict(rows=-1), dict(max_q=0, cu=P16), dict(pages=0),
               dict(n_pages=0), dict(window=-1), dict(window=4, causal=0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(pages=1 << 27),  # 64 x 2^27 positions
               dict(rows=3), dict(max_q=2), dict(rows=1 << 30, cu=P16), dict(qv=_view(row=-8))]:
        assert _attn(lib, **kw) == -3, kw
    for kw in [dict(qv=None), dict(qv=_view(None)), dict(table=None), dict(lens=None), dict(pool=None), dict(out=None),
               dict(ws=None), dict(err=None)]:
        assert _attn(lib, **kw) == -1, kw
    odd = ctypes.c_void_p(16 * 1024 + 4)
    for kw in [dict(qv=_view(odd)), dict(qv=_view(head=12)), dict(pool=odd), dict(out=odd), dict(ws=odd),
               dict(lse=ctypes.c_void_p(16 * 1024 + 2))]:
        assert _attn(lib, **kw) == -4, kw
    assert _attn(lib, out=P16) == -3                      # over the queries
    assert _attn(lib, out=PFAR, lse=PFAR) == -3


def _append_bf16(lib, B=2, rows=2, kv=P16, stride=576, cu=P16, lens=P16, nxt=None, max_new=1, w=None, eps=1e-6, rot=None, qv=None,
                 heads=0, q_out=None, c=None, kr=None, table=P16, pages=4, P=64, pool=PFAR, n_pages=4, err=P16):
    return lib.mla_qcache_append_bf16(B, rows, kv, stride, cu, lens, nxt, max_new, w, ctypes.c_float(eps), rot, qv, heads, q_out, c,
                                      kr, table, pages, P, pool, n_pages, err, None)


def test_append_bf16_refusals(lib):
    assert _append_bf16(lib, rows=0) == 0
    assert _append_bf16(lib, P=16) == -2
    for kw in [dict(B=0), dict(rows=-1), dict(max_new=0), dict(pages=0), dict(n_pages=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(stride=-576), dict(rot=_rot(dim=128)), dict(rot=_rot(dim=8)), dict(c=P16), dict(c=PFAR)]:
        assert _append_bf16(lib, **kw) == -3, kw
    for kw in [dict(kv=None), dict(cu=None), dict(lens=None), dict(table=None), dict(err=None), dict(pool=None),
               dict(q_out=PFAR), dict(qv=_view(), heads=4)]:
        assert _append_bf16(lib, **kw) == -1, kw
    for kw in [dict(kv=ctypes.c_void_p(16 * 1024 + 4)), dict(stride=580), dict(w=ctypes.c_void_p(16 * 1024 + 2)),
               dict(pool=ctypes.c_void_p((1 << 40) + 8))]:
        assert _append_bf16(lib, **kw) == -4, kw


def test_binding_refuses_host_tensors(lib):
    cfg = q.make_kv4_config(8)
    z = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(q.QCacheError, match="CUDA"):
        q.mla_qcache_kv4_attn(cfg, z, i.view(1, 1), i, z, 1.0, z, z, i)
    with pytest.raises(q.QCacheError, match="CUDA"):
        q.mla_qcache_kv4_append(cfg, z, z, i, i, 1, i, z, i)
    with pytest.raises(q.QCacheError, match="CUDA"):
        q.mla_qcache_append_bf16(z, i, i, 1, i, z, i)
    with pytest.raises(q.QCacheError, match="required"):
        q.mla_qcache_kv4_attn(cfg, None, i, i, z, 1.0, z, z, i)
    with pytest.raises(TypeError):
        q.mla_qcache_kv4_attn(cfg, 3, i, i, z, 1.0, z, z, i)

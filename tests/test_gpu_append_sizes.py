"""Both appends at the row counts where another form of the kernel takes over (2048 rows) and with more sequences than one
load per lane finds (32), against the plain statements: every output, and the rows behind the last sequence."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import kv4_ref as ref
from tests.test_gpu_append_bf16 import near
from tests.test_gpu_kv4 import TYPES, error_word, ints, offsets, tables

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def batch(rng, B, rows, P):
    """Rows of B sequences, empty ones among them, behind lengths of their own; a table with pages to spare."""
    cuts = np.sort(rng.integers(0, rows + 1, B - 1))
    new = np.diff(np.concatenate([[0], cuts, [rows]]))
    new[rng.integers(0, B, B // 5)] = 0
    new[int(rng.integers(0, B))] += rows - new.sum()
    base = rng.integers(0, 3 * P, B)
    pages = -(-int((base + new).max()) // P)
    table = rng.permutation(B * pages).astype(np.int32).reshape(B, pages)
    seq = np.repeat(np.arange(B), new)
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(base, new)])
    return new, base, table, seq, pos


@pytest.mark.parametrize("rows,B,Hkv,Hq,D,group,P,dtype,rot,interleaved", [
    (2047, 3, 3, 21, 128, 64, 32, "bf16", 128, False), (2048, 40, 1, 1, 128, 128, 64, "fp16", 128, True),
    (2049, 33, 5, 10, 64, 32, 16, "bf16", 48, False), (5003, 300, 1, 3, 64, 64, 16, "fp16", 64, False),
    (2051, 1, 5, 5, 128, 32, 256, "bf16", 64, True), (3001, 32, 3, 0, 128, 128, 128, "bf16", 0, False),
    (70, 64, 3, 21, 128, 128, 16, "bf16", 128, False), (64, 64, 2, 14, 64, 64, 32, "fp16", 64, True)])
def test_grouped_query_append(rows, B, Hkv, Hq, D, group, P, dtype, rot, interleaved):
    rng, t, pad = np.random.default_rng(rows + B), TYPES[dtype], 5
    cfg = q.make_kv4_config(Hkv, D, group=group, page_size=P)
    if rows == B:  # a decode step: one row each
        new, base = np.ones(B, int), rng.integers(0, 3 * P, B)
        table = rng.permutation(B * 4).astype(np.int32).reshape(B, 4)
        seq, pos = np.arange(B), base
    else:
        new, base, table, seq, pos = batch(rng, B, rows, P)
    qkv = torch.tensor(rng.standard_normal((rows + pad, Hq + 2 * Hkv, D), dtype=np.float32) * np.exp(rng.standard_normal((1, 1, D))),
                       dtype=torch.float32).to(t).cuda()
    cos, sin = tables(int(pos.max()) + 1, rot) if rot else (None, None)
    angles = dict(cos=torch.tensor(cos).cuda(), sin=torch.tensor(sin).cuda()) if rot else {}
    pool = torch.randint(0, 256, (table.size, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    want = pool.cpu().numpy().copy()
    mark = lambda *s: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    q_out, kd, vd, nxt, err = mark(rows + pad, Hq, D), mark(rows + pad, Hkv, D), mark(rows + pad, Hkv, D), ints([-1] * B), error_word()
    q.mla_qcache_kv4_append(cfg, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], offsets(new), ints(base), int(new.max()), ints(table), pool, err,
                            interleaved=interleaved, q=qkv[:, :Hq] if Hq else None, q_out=q_out if Hq else None, k_deq=kd, v_deq=vd,
                            seq_lens_next=nxt, **angles)
    torch.cuda.synchronize()
    assert int(err) == 0 and np.array_equal(nxt.cpu().numpy(), base + new)
    x = qkv[:rows].float().cpu().numpy()
    qk = ref.rotate32(x[:, :Hq + Hkv], cos[pos], sin[pos], interleaved) if rot else x[:, :Hq + Hkv]
    kq, vq = ref.quantize(qk[:, Hq:].astype(np.float64), group), ref.quantize(x[:, Hq + Hkv:].astype(np.float64), group)
    pages, at = want.reshape(table.size, Hkv, -1), (table[seq, pos // P], slice(None), pos % P)
    regions = [(0, D // 2), (P * D // 2, D // 2), (P * D, 8 * (D // group))]
    numbers = np.ascontiguousarray(np.stack([kq[1], kq[2], vq[1], vq[2]], -1).astype(np.float16))
    for (begin, width), data in zip(regions, (ref.pack_rows(kq[0], ref.key_nibble, D), ref.pack_rows(vq[0], ref.value_nibble, D),
                                              numbers.view(np.uint8).reshape(rows, Hkv, -1))):
        view = np.lib.stride_tricks.as_strided(pages[:, :, begin:], (table.size, Hkv, P, width), (*pages.strides[:2], width, 1))
        view[at] = data
    assert np.array_equal(pool.cpu().numpy(), want)
    same = lambda got, exp: torch.equal(got[:rows].cpu(), torch.tensor(np.float32(exp)).to(t))  # noqa: E731
    assert same(kd, ref.values(*kq, group)) and same(vd, ref.values(*vq, group)) and (not Hq or same(q_out, qk[:, :Hq]))
    for o in (q_out, kd, vd):
        assert (o[rows:] == 7).all()


@pytest.mark.parametrize("rows,B,H,P,interleaved,norm,rot", [
    (2047, 3, 3, 64, True, True, 64), (2048, 40, 1, 32, False, True, 64), (2049, 33, 21, 128, True, True, 64), (2050, 1, 16, 64, False, False, 32),
    (2051, 300, 5, 32, True, True, 0), (5003, 32, 0, 128, False, True, 64), (70, 64, 21, 32, True, True, 64), (64, 64, 128, 64, False, True, 64)])
def test_latent_append(rows, B, H, P, interleaved, norm, rot):
    rng, pad = np.random.default_rng(rows + B), 5
    if rows == B:
        new, base = np.ones(B, int), rng.integers(0, 3 * P, B)
        table = rng.permutation(B * 4).astype(np.int32).reshape(B, 4)
        seq, pos = np.arange(B), base
    else:
        new, base, table, seq, pos = batch(rng, B, rows, P)
    gen = lambda *s: torch.tensor(rng.standard_normal(s, dtype=np.float32)).to(BF).cuda()  # noqa: E731
    kv, qfull = (3 * gen(rows + pad, 640))[:, :576], gen(rows + pad, max(1, H), 192)
    weight = 1 + gen(512) * 0.2 if norm else None
    cos, sin = tables(int(pos.max()) + 1, rot) if rot else (None, None)
    angles = dict(cos=torch.tensor(cos).cuda(), sin=torch.tensor(sin).cuda()) if rot else {}
    pool = gen(table.size, P, 576)
    want = pool.clone()
    mark = lambda *s: torch.full(s, 7.0, dtype=BF, device="cuda")  # noqa: E731
    q_out, c_out, kr_out, nxt, err = mark(rows + pad, H, 64), mark(rows + pad, 512), mark(rows + pad, 64), ints([-1] * B), error_word()
    q.mla_qcache_append_bf16(kv, offsets(new), ints(base), int(new.max()), ints(table), pool, err, norm_weight=weight, eps=1e-5,
                             interleaved=interleaved, q_rope=qfull[..., 128:] if H else None, q_out=q_out if H else None, c_out=c_out,
                             kr_out=kr_out, seq_lens_next=nxt, **angles)
    torch.cuda.synchronize()
    assert int(err) == 0 and np.array_equal(nxt.cpu().numpy(), base + new)
    c = kv[:rows, :512].double().cpu().numpy()
    if norm:
        c = c / np.sqrt((c * c).mean(-1, keepdims=True) + float(np.float32(1e-5))) * weight.double().cpu().numpy()
        assert near(c_out[:rows], c).all()
    else:
        assert torch.equal(c_out[:rows], kv[:rows, :512])
    heads = torch.cat([kv[:rows, None, 512:], qfull[:rows, :H, 128:]], 1).float().cpu().numpy()
    turned = torch.tensor(ref.rotate32(heads, cos[pos], sin[pos], interleaved) if rot else heads).to(BF).cuda()
    assert torch.equal(kr_out[:rows], turned[:, 0]) and torch.equal(q_out[:rows], turned[:, 1:])
    place = torch.tensor(table[seq, pos // P].astype(np.int64)).cuda(), torch.tensor(pos % P).cuda()
    want[place] = torch.cat([c_out[:rows], kr_out[:rows]], -1)
    assert torch.equal(pool, want)
    for o in (q_out, c_out, kr_out):
        assert (o[rows:] == 7).all()


@pytest.mark.parametrize("D,group", [(128, 128), (64, 32)])
def test_what_the_cache_holds_for_groups_that_are_reported(D, group):
    """Finite numbers: zeros for an infinity or for no number at all, the minimum for a NaN among numbers, the end of the
    range beyond it; the groups beside them as ever."""
    cfg, rng = q.make_kv4_config(1, D, group=group, page_size=16), np.random.default_rng(D)
    x = rng.standard_normal((8, 1, D)).astype(np.float32)
    x = torch.tensor(x).bfloat16().float().numpy()
    plain = ref.quantize(x.astype(np.float64), group)
    want = ref.values(*plain, group)
    x[0, 0, :group], x[1, 0, 3], x[2, 0, :group] = np.nan, np.nan, np.inf
    x[3, 0, 5], x[4, 0, 6] = -np.inf, 3e38
    x[5, 0, :group], x[6, 0, 2] = -1e6, 70000.0
    want[[0, 2], :, :group] = want[3, :, :group] = 0
    kv = torch.tensor(x).bfloat16().cuda()
    pool, err = torch.zeros((1, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda"), error_word()
    kd, vd = torch.empty_like(kv), torch.empty_like(kv)
    q.mla_qcache_kv4_append(cfg, kv, kv, ints([0, 8]), ints([0]), 8, ints([[0]]), pool, err, k_deq=kd, v_deq=vd)
    assert int(err) == q.DEV_NONFINITE | q.DEV_RANGE
    k, v, _, _ = ref.read_sequence(pool.cpu().numpy(), np.array([0]), 8, 1, D, group, 16)
    assert np.array_equal(k, v) and np.isfinite(k).all() and np.abs(k).max() <= 65504
    assert torch.equal(kd.cpu(), torch.tensor(k[0, :, None]).float().bfloat16()) and torch.equal(kd, vd)
    k = k[0, :, None]
    for r in (0, 2, 3, 7):
        assert np.array_equal(k[r], want[r]), r
    assert np.array_equal(k[:, :, group:], want[:, :, group:])
    rest = np.arange(group) != 3
    assert np.abs(k[1, 0, :group][rest] - x[1, 0, :group][rest]).max() <= (x[1, 0, :group][rest].max() - x[1, 0, :group][rest].min()) / 29
    assert k[1, 0, 3] == k[1, 0, :group].min()  # (the minimum level itself may be held by no other)
    assert (k[5, 0, :group] == -65504).all() and k[4, 0, 6] > 60000 and k[6, 0, 2] > 60000

"""Append to the paged BF16 latent cache on the GPU: norm, rotation and placement against the plain statement in
64 bits, and runs in front of the operators that read its results (the unquantized decode, the packed writer)."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
import oracle
import workloads
from tests import gpu_util as gu
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import error_word, ints, offsets, tables

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def near(got, want):
    """BF16 results of float32 arithmetic: half a step of the result, plus the arithmetic's error (a norm over 512
    squares and a few products, or a difference of two products: below 2^-16 of the terms)."""
    got = got.double().cpu().numpy()
    return np.abs(got - want) <= 2.0 ** -9 * 2 * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -16 * (np.abs(want) + 1e-30)


@pytest.mark.parametrize("P,H,interleaved,norm,rot", [(64, 16, True, True, 64), (32, 3, False, True, 64), (128, 1, True, False, 64),
                                                      (64, 128, False, True, 32), (32, 5, True, True, 0)])
def test_rows_norm_rotation_and_place(P, H, interleaved, norm, rot):
    rng = np.random.default_rng(P + H)
    base, new, pad = [0, P - 1, 2 * P, 7], [3, P + 1, 0, 1], 2
    B, rows, pages = 4, sum(new), 4
    table = rng.permutation(B * pages).astype(np.int32).reshape(B, pages)
    wide = torch.tensor(rng.standard_normal((rows + pad, 640)) * 3, dtype=torch.float32).to(BF).cuda()  # rows with a stride
    kv = wide[:, :576]
    qfull = torch.tensor(rng.standard_normal((rows + pad, H, 192)), dtype=torch.float32).to(BF).cuda()
    weight = torch.tensor(1 + 0.2 * rng.standard_normal(512), dtype=torch.float32).to(BF).cuda() if norm else None
    cos, sin = tables(3 * P + 8, rot) if rot else (None, None)
    pool = torch.tensor(rng.standard_normal((B * pages, P, 576)), dtype=torch.float32).to(BF).cuda()
    before = pool.clone()
    mark = lambda *s: torch.full(s, 7.0, dtype=BF, device="cuda")  # noqa: E731
    q_out, c_out, kr_out = mark(rows + pad, H, 64), mark(rows + pad, 512), mark(rows + pad, 64)
    nxt, err = ints([0] * B), error_word()
    q.mla_qcache_append_bf16(kv, offsets(new), ints(base), max(new), ints(table), pool, err, norm_weight=weight, eps=1e-5,
                             cos=torch.tensor(cos).cuda() if rot else None, sin=torch.tensor(sin).cuda() if rot else None,
                             interleaved=interleaved, q_rope=qfull[..., 128:], q_out=q_out, c_out=c_out, kr_out=kr_out, seq_lens_next=nxt)
    torch.cuda.synchronize()
    assert int(err) == 0 and nxt.tolist() == [b + n for b, n in zip(base, new)]
    x = kv[:rows].double().cpu().numpy()
    c = x[:, :512]
    if norm:
        c = c / np.sqrt((c * c).mean(-1, keepdims=True) + float(np.float32(1e-5))) * weight.double().cpu().numpy()
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(base, new)])
    seq = np.repeat(np.arange(B), new)
    heads = torch.cat([kv[:rows, None, 512:], qfull[:rows, :, 128:]], 1).float().cpu().numpy()
    turned = ref.rotate32(heads, cos[pos], sin[pos], interleaved) if rot else heads
    turned = torch.tensor(turned).to(BF)
    if norm:
        assert near(c_out[:rows], c).all()
    else:
        assert torch.equal(c_out[:rows], kv[:rows, :512])
    assert torch.equal(kr_out[:rows].cpu(), turned[:, 0]) and torch.equal(q_out[:rows].cpu(), turned[:, 1:])
    want = before.clone()
    for r in range(rows):
        want[int(table[seq[r], pos[r] // P]), int(pos[r] % P)] = torch.cat([c_out[r], kr_out[r]])
    assert torch.equal(pool, want)
    for o in (q_out, c_out, kr_out):
        assert (o[rows:] == 7).all()
    # rows alone, without a pool
    c2, k2 = mark(rows + pad, 512), mark(rows + pad, 64)
    q.mla_qcache_append_bf16(kv, offsets(new), ints(base), max(new), None, None, err, norm_weight=weight, eps=1e-5,
                             cos=torch.tensor(cos).cuda() if rot else None, sin=torch.tensor(sin).cuda() if rot else None,
                             interleaved=interleaved, c_out=c2, kr_out=k2)
    assert torch.equal(c2, c_out) and torch.equal(k2, kr_out) and int(err) == 0


def test_reports_what_it_skips():
    kv = torch.randn(3, 576, device="cuda").to(BF)

    def run(cu, lens, table, max_new=3):
        pool = torch.zeros((3, 32, 576), dtype=BF, device="cuda")
        err = error_word()
        q.mla_qcache_append_bf16(kv, ints(cu), ints(lens), max_new, ints(table), pool, err)
        return int(err), int((pool != 0).any(-1).sum())
    assert run([0, 1, 3], [0, 0], [[0], [1]]) == (0, 3)
    assert run([0, 1, 3], [0, 0], [[0], [3]]) == (q.DEV_BAD_PAGE, 1)
    assert run([0, 1, 3], [32, 0], [[0], [1]]) == (q.DEV_SEQ_OVERFLOW, 2)
    assert run([0, 1, 3], [0, 0], [[0], [1]], max_new=1) == (q.DEV_ROWS, 1)
    assert run([0, 1, 2], [0, 0], [[0], [1]]) == (0, 2)  # a padded row


def test_append_then_unquantized_decode():
    """Raw rows -> append -> mla_qcache_decode_attn_bf16, against the oracle's attention over the same rows."""
    rng = np.random.default_rng(4)
    B, H, P, pages, lens = 2, 16, 64, 4, [150, 37]
    kv = torch.tensor(rng.standard_normal((sum(lens), 576)), dtype=torch.float32).to(BF).cuda()
    qr = torch.tensor(rng.standard_normal((sum(lens), H, 64)), dtype=torch.float32).to(BF).cuda()
    weight = torch.ones(512, dtype=BF, device="cuda")
    cos, sin = (torch.tensor(x).cuda() for x in tables(256, 64))
    table = rng.permutation(B * pages).astype(np.int32).reshape(B, pages)
    pool = torch.zeros((B * pages, P, 576), dtype=BF, device="cuda")
    lens_d, err, q_out = ints([0] * B), error_word(), torch.empty_like(qr)
    nxt = ints([0] * B)
    q.mla_qcache_append_bf16(kv, offsets(lens), lens_d, max(lens), ints(table), pool, err, norm_weight=weight, cos=cos, sin=sin,
                             interleaved=True, q_rope=qr, q_out=q_out, seq_lens_next=nxt)
    last = torch.tensor([lens[0] - 1, sum(lens) - 1], device="cuda")
    q_lat = torch.tensor(rng.standard_normal((B, H, 512)), dtype=torch.float32).to(BF).cuda()
    q_rope = q_out[last].contiguous()
    out, lse = torch.empty((B, H, 512), device="cuda"), torch.empty((B, H), device="cuda")
    ws = torch.zeros(q.bf16_workspace_bytes(B, H, pages, P), dtype=torch.uint8, device="cuda")
    q.mla_qcache_decode_attn_bf16(q_lat, q_rope, ints(table), P, nxt, pool, 0.07, out, lse, ws, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    o, l, fl = oracle.decode_bf16(bits(q_lat), bits(q_rope), table, P, np.array(lens, np.int32), bits(pool), 0.07)
    assert fl == 0
    gu.check_decode(out, lse, o, l)


def test_rows_feed_the_packed_writer():
    """c_out and kr_out are the packed writer's inputs: its BF16 buffers and pages hold what the oracle's do for them."""
    w = workloads.Workload("feed", 2, 16, 1, 4, 64, seed=3)
    inp = workloads.make_inputs(w, seq_lens=np.array([130, 70], np.int32))
    rows = int(inp.cu[-1])
    kv = torch.randn(rows, 576, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    weight = torch.ones(512, dtype=BF, device="cuda")
    cos, sin = (torch.tensor(x).cuda() for x in tables(256, 64))
    c, kr, err = torch.empty(rows, 512, dtype=BF, device="cuda"), torch.empty(rows, 64, dtype=BF, device="cuda"), error_word()
    q.mla_qcache_append_bf16(kv, ints(inp.cu), ints([0, 0]), 130, None, None, err, norm_weight=weight, cos=cos, sin=sin, interleaved=True,
                             c_out=c, kr_out=kr)
    cache = gu.gpu_cache(w.config_kwargs(), inp)
    cache.write(c, kr, ints(inp.cu), 130)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ocfg, pool, sink, ring = gu.oracle_cache(w.config_kwargs(), inp)
    assert oracle.write(ocfg, bits(c), bits(kr), inp.cu, np.zeros(2, np.int32), 130, inp.page_table, pool, sink, ring) == 0
    gu.assert_cache_equal(cache, pool, sink, ring)
    assert int(err) == 0 and cache.error_bits() == 0

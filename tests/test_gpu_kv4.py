"""Grouped-query cache in 4 bits on the GPU against the plain statement in 64 bits (kv4_ref): the append byte
for byte, the attention within the bound that its arithmetic gives, at the sizes, masks and layouts where it
can go wrong; then runs of both as a decoder uses them."""
import math

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import kv4_ref as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ints(v):
    return torch.tensor(np.asarray(v), dtype=I32, device="cuda")


def offsets(n):
    return ints(np.concatenate([[0], np.cumsum(n)]))


def tables(n_pos, rot):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None]
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def error_word():
    return torch.zeros(1, dtype=I32, device="cuda")


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("D,group,P,Hkv,Hq,dtype,rot,interleaved", [
    (128, 128, 64, 2, 8, "bf16", 128, False), (128, 64, 16, 3, 3, "fp16", 128, True), (128, 32, 128, 1, 7, "bf16", 64, False),
    (64, 64, 32, 5, 10, "fp16", 64, False), (64, 32, 16, 2, 14, "bf16", 32, True), (128, 128, 256, 4, 4, "bf16", 0, False),
    (64, 64, 64, 8, 64, "bf16", 48, False), (128, 64, 32, 1, 1, "fp16", 16, True)])
def test_append_is_the_plain_statement_byte_for_byte(D, group, P, Hkv, Hq, dtype, rot, interleaved):
    rng = np.random.default_rng(D + group + P + rot)
    t = TYPES[dtype]
    cfg = q.make_kv4_config(Hkv, D, group=group, page_size=P)
    base, new = [0, P - 1, 2 * P + 3, 5], [1, 2, 0, P + 2]  # an empty cache, over a page's end, nothing new, a whole page and more
    B, rows, pad = 4, sum(new), 3
    pages = 5
    table = rng.permutation(B * pages).astype(np.int32).reshape(B, pages)
    # one projection's output: q | k | v of each row, then rows of a padded batch
    qkv = torch.tensor(rng.standard_normal((rows + pad, Hq + 2 * Hkv, D)) * np.exp(rng.standard_normal((1, 1, D))), dtype=torch.float32)
    qkv[0, Hq:] = 0.75   # a constant key and value: scale 0
    qkv = qkv.to(t).cuda()
    cos, sin = tables(max(b + n for b, n in zip(base, new)), rot) if rot else (None, None)
    pool = torch.randint(0, 256, (B * pages, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    want = pool.cpu().numpy().copy()
    mark = lambda *s: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    q_out, kd, vd = mark(rows + pad, Hq, D), mark(rows + pad, Hkv, D), mark(rows + pad, Hkv, D)
    lens, nxt, err = ints(base), ints([-1] * B), error_word()
    q.mla_qcache_kv4_append(cfg, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], offsets(new), lens, max(new), ints(table), pool, err,
                            cos=None if cos is None else torch.tensor(cos).cuda(), sin=None if sin is None else torch.tensor(sin).cuda(),
                            interleaved=interleaved, q=qkv[:, :Hq], q_out=q_out, k_deq=kd, v_deq=vd, seq_lens_next=nxt)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert nxt.tolist() == [b + n for b, n in zip(base, new)] and lens.tolist() == base
    x = qkv.float().cpu().numpy()
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(base, new)])
    seq = np.repeat(np.arange(B), new)
    qk = ref.rotate32(x[:rows, :Hq + Hkv], cos[pos], sin[pos], interleaved) if rot else x[:rows, :Hq + Hkv]
    kq = ref.quantize(qk[:, Hq:].astype(np.float64), group)
    vq = ref.quantize(x[:rows, Hq + Hkv:].astype(np.float64), group)
    for r in range(rows):
        for h in range(Hkv):
            ref.put_token(want, table[seq[r], pos[r] // P], pos[r] % P, h, D, group, P, [a[r, h] for a in kq], [a[r, h] for a in vq])
    assert np.array_equal(pool.cpu().numpy(), want)
    same = lambda got, exp: torch.equal(got[:rows].cpu(), torch.tensor(np.float32(exp)).to(t))  # noqa: E731
    assert same(q_out, qk[:, :Hq])
    assert same(kd, ref.values(*kq, group)) and same(vd, ref.values(*vq, group))
    for o in (q_out, kd, vd):  # rows behind the last sequence stay
        assert (o[rows:] == 7).all()


def test_append_codes_at_the_borders_between_levels():
    """Values on, just below and just above the midpoints of the levels: exact ties go to the even code."""
    D = 128
    cfg = q.make_kv4_config(1, D, page_size=16)
    n = 64
    x = np.zeros((n, 1, D), np.float32)
    rng = np.random.default_rng(3)
    for r in range(n):
        e = 2.0 ** rng.integers(-6, 6)
        mids = (np.arange(15) + 0.5) * e
        x[r, 0, 0], x[r, 0, 1] = 0, 15 * e
        x[r, 0, 2:17] = mids
        x[r, 0, 17:32] = mids * (1 - 2.0 ** -8)
        x[r, 0, 32:47] = mids * (1 + 2.0 ** -7)
        x[r] -= e * rng.integers(0, 8)
    k = torch.tensor(x).bfloat16().cuda()
    pool = torch.zeros((4, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    err = error_word()
    q.mla_qcache_kv4_append(cfg, k, k, ints([0, n]), ints([0]), n, ints([[0, 1, 2, 3]]), pool, err)
    codes, s, m = ref.quantize(k.double().cpu().numpy(), D)
    want = np.zeros(pool.shape, np.uint8)
    for r in range(n):
        kv = [a[r, 0] for a in (codes, s, m)]
        ref.put_token(want, r // 16, r % 16, 0, D, D, 16, kv, kv)
    assert np.array_equal(pool.cpu().numpy(), want) and int(err) == 0


def test_append_reports_what_it_skips():
    cfg = q.make_kv4_config(2, 64, page_size=16)
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()

    def run(cu, lens, table, max_new=4, k=k, n_pos=None):
        pool = torch.zeros((4, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
        err = error_word()
        ang = None if n_pos is None else torch.ones(n_pos, 32, device="cuda")
        q.mla_qcache_kv4_append(cfg, k, k, ints(cu), ints(lens), max_new, ints(table), pool, err, cos=ang, sin=ang)
        return int(err), int((pool != 0).any(1).sum())
    assert run([0, 1, 4], [0, 0], [[0], [1]]) == (0, 2)
    assert run([0, 1, 4], [0, 0], [[0], [9]]) == (q.DEV_BAD_PAGE, 1)
    assert run([0, 1, 4], [0, 0], [[-1], [1]]) == (q.DEV_BAD_PAGE, 1)
    assert run([0, 1, 4], [16, 0], [[0], [1]]) == (q.DEV_SEQ_OVERFLOW, 1)
    assert run([0, 1, 4], [-3, 0], [[0], [1]]) == (q.DEV_SEQ_OVERFLOW, 1)
    assert run([0, 1, 4], [0, 0], [[0], [1]], max_new=2) == (q.DEV_ROWS, 1)
    assert run([0, 1, 4], [5, 0], [[0], [1]], n_pos=5) == (q.DEV_SEQ_OVERFLOW, 1)  # no angle for position 5
    bad = k.clone()
    bad[2, 1, 5] = float("nan")
    assert run([0, 1, 4], [0, 0], [[0], [1]], k=bad)[0] == q.DEV_NONFINITE
    bad[2, 1, 5] = 3e38
    assert run([0, 1, 4], [0, 0], [[0], [1]], k=bad)[0] == q.DEV_RANGE
    # scale and minimum fit FP16; the top level does (scale 8704: 65280) or not (scale 8733.87 -> 8736: 65536)
    for top, word in ((65280.0, 0), (65504.0, q.DEV_RANGE)):
        f16 = torch.zeros(4, 2, 64, device="cuda").half()
        f16[2, 1, 5], f16[2, 1, 6] = top, -top
        assert run([0, 1, 4], [0, 0], [[0], [1]], k=f16)[0] == word


# ---------------------------------------------------------------- attention
class Case:
    """A cache of random tokens (written by the append) and queries; lens: tokens, new: query rows of each."""

    def __init__(self, lens, new, Hkv=2, G=4, D=128, group=None, P=16, dtype="bf16", seed=0, pad=0, spare=1, loud=1.0, n_pages=None):
        rng = np.random.default_rng(seed)
        self.t, self.lens, self.new = TYPES[dtype], list(lens), list(new)
        self.cfg = q.make_kv4_config(Hkv, D, group=group, page_size=P)
        self.D, self.P, self.group, self.Hkv, self.Hq, self.pad = D, P, group or D, Hkv, Hkv * G, pad
        B, total = len(lens), sum(lens)
        pages = max(1, -(-max(lens) // P)) + spare
        self.n_pages = n_pages or B * pages
        self.table = rng.permutation(self.n_pages)[:B * pages].astype(np.int32).reshape(B, pages)
        self.pool = torch.full((self.n_pages, q.kv4_page_bytes(self.cfg)), 0xFF, dtype=torch.uint8, device="cuda")  # NaN numbers
        self.err = error_word()
        if total:
            kv = torch.tensor(rng.standard_normal((2, total, Hkv, D)) * loud, dtype=torch.float32).to(self.t).cuda()
            q.mla_qcache_kv4_append(self.cfg, kv[0], kv[1], offsets(lens), ints([0] * B), max(lens), ints(self.table), self.pool, self.err)
        self.q = torch.tensor(rng.standard_normal((sum(new) + pad, self.Hq, D)) * 2, dtype=torch.float32).to(self.t).cuda()

    def workspace(self, max_q=None):
        n = q.kv4_workspace_bytes(self.cfg, len(self.lens), self.Hq, max_q or max(1, max(self.new)), self.table.shape[1])
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def run(self, scale=None, window=0, causal=True, lse=True, ws=None, max_q=None, one=False, qq=None, out=None, stream=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        rows = sum(self.new) + self.pad
        out = torch.full((rows, self.Hq, self.D), 7.0, dtype=self.t, device="cuda") if out is None else out
        l = torch.full((rows, self.Hq), 7.0, device="cuda") if lse else None
        max_q = max_q or max(1, max(self.new))
        q.mla_qcache_kv4_attn(self.cfg, self.q if qq is None else qq, ints(self.table), ints(self.lens), self.pool, scale, out,
                              self.workspace(max_q) if ws is None else ws, self.err, cu_q=None if one else offsets(self.new),
                              max_q=max_q, lse=l, causal=causal, window=window, stream=stream)
        return out, l

    def check(self, scale=None, window=0, causal=True, lse=True, **kw):
        out, l = self.run(scale, window, causal, lse, **kw)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        pool, r = self.pool.cpu().numpy(), 0
        tensor_rows = max(1, max(self.new)) * (self.Hq // self.Hkv) > 16
        for b, (T, n) in enumerate(zip(self.lens, self.new)):
            k, v, vs, most = ref.read_sequence(pool, self.table[b], T, self.Hkv, self.D, self.group, self.P)
            qq = self.q[r:r + n].double().cpu().numpy()
            ok = ref.seen(T, n, causal, window)
            want, wl, bound = ref.attention(qq, k, v, vs, most, scale, ok, self.t, tensor_rows)
            got = out[r:r + n].double().cpu().numpy()
            assert np.isfinite(got).all()
            worst = (np.abs(got - want) - bound).max(initial=-1)
            assert worst <= 0, f"sequence {b} (T={T}, n={n}): off by {worst:.3e} more than its bound"
            if lse:
                gl = l[r:r + n].double().cpu().numpy()
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
                fin = np.isfinite(wl)
                lb = ref.lse_bound(qq, k, scale, ok)
                assert (np.abs(gl[fin] - wl[fin]) <= lb[fin]).all(), np.abs(gl[fin] - wl[fin]).max()
            r += n
        if self.pad:  # rows behind the last sequence stay
            assert (out[r:] == 7).all() and (not lse or (l[r:] == 7).all())
        return out, l


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300])
def test_single_token_lengths(T):
    Case([T, 1, T + 1], [1, 1, 1], P=16, seed=T).check(one=True)


@pytest.mark.parametrize("D,group,P,Hkv,G,dtype", [
    (128, 128, 64, 2, 1, "bf16"), (128, 64, 16, 1, 8, "fp16"), (128, 32, 32, 3, 5, "bf16"), (64, 64, 128, 2, 7, "fp16"),
    (64, 32, 16, 4, 2, "bf16"), (128, 128, 256, 1, 16, "bf16"), (128, 64, 64, 2, 12, "fp16"), (64, 64, 16, 1, 9, "bf16"),
    (128, 32, 16, 1, 16, "fp16"), (64, 32, 64, 2, 11, "fp16")])
def test_single_token_layouts(D, group, P, Hkv, G, dtype):
    Case([257, 40, 3], [1, 1, 1], Hkv=Hkv, G=G, D=D, group=group, P=P, dtype=dtype, seed=D + G).check()


@pytest.mark.parametrize("D,group,G,dtype,n", [
    (128, 128, 4, "bf16", 5), (128, 64, 8, "fp16", 16), (64, 64, 7, "bf16", 19), (64, 32, 4, "fp16", 33), (128, 32, 1, "bf16", 17),
    (128, 128, 8, "fp16", 40), (64, 64, 16, "bf16", 9), (128, 64, 5, "bf16", 60)])
@pytest.mark.parametrize("lse", [True, False])
def test_many_rows(D, group, G, dtype, n, lse):
    """One tile of queries (up to 128 rows) and two (more); drafted tokens and prompts from an empty cache."""
    Case([n, n + 1, 200 + n, 131], [n, n, n, 3], Hkv=2, G=G, D=D, group=group, P=16, dtype=dtype, seed=n + G).check(lse=lse)


@pytest.mark.parametrize("n,G,D,group,P", [
    (17, 1, 128, 128, 16), (5, 5, 128, 64, 256), (8, 4, 64, 32, 64), (32, 1, 128, 32, 128), (33, 1, 128, 128, 256), (12, 5, 64, 64, 16),
    (16, 4, 128, 32, 32), (13, 5, 128, 64, 64), (32, 4, 64, 32, 128), (43, 3, 128, 32, 256), (37, 7, 64, 64, 256)])
@pytest.mark.parametrize("window", [0, 130])
def test_row_counts_at_the_borders_between_kernels(n, G, D, group, P, window):
    """Up to 32 rows (two blocks of 16), up to 64, up to 128, more; sequences cut over the SMs, ends inside a page and a tile."""
    Case([n, 700, 1201, 300], [n, n, 1, 2], Hkv=2, G=G, D=D, group=group, P=P, dtype="fp16" if n & 1 else "bf16", seed=n + D).check(window=window)


def test_rows_of_several_blocks_and_more_items_than_the_gpu_holds():
    Case([400], [300], Hkv=1, G=4, seed=1).check(lse=False)          # five blocks of 256 rows, cut over the SMs
    Case([40] * 160, [20] * 160, Hkv=2, G=1, seed=2, D=64).check()   # 320 items: one CTA each


@pytest.mark.parametrize("n,G", [(1, 2), (5, 8), (20, 4)])
def test_many_sequences(n, G):
    """More sequences than the quick ways of sharing the work hold; a few long ones among many that are short or empty."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 20, 700)
    lens[[3, 350, 699]] = [300, 90, 150]
    new = np.minimum(rng.integers(0, n + 1, 700), lens)
    c = Case(lens.tolist(), new.tolist(), Hkv=1, G=G, D=64, P=16, seed=n, pad=3)
    c.check(max_q=n)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 40, 100, 1000])
@pytest.mark.parametrize("n,G", [(1, 3), (5, 2), (30, 4)])
def test_sliding_window(window, n, G):
    Case([n, 150, 201], [n, n, min(n, 7)], G=G, seed=window).check(window=window)


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("n,G", [(1, 4), (5, 3), (6, 4), (12, 4), (30, 4), (70, 4)])
def test_pages_behind_the_window_may_be_gone(n, G, P):
    """A loop that frees the pages behind its window leaves any id there; steps and tiles of a kernel begin before the window."""
    window = 100
    c = Case([n, 700, 450], [n, n, min(n, 3)], G=G, P=P, seed=n + P)
    full = c.table.copy()
    a, l = c.check(window=window)
    for b, (T, m) in enumerate(zip(c.lens, c.new)):
        c.table[b, :max(0, T - m - window + 1) // P] = -1
    b, k = c.run(window=window)
    torch.cuda.synchronize()
    assert (c.table != full).any() and int(c.err) == 0
    assert torch.equal(a, b) and torch.equal(l, k)


@pytest.mark.parametrize("n,G", [(1, 4), (3, 5), (24, 3)])
def test_rows_that_see_nothing(n, G):
    """More query rows than tokens, and an empty cache: those rows give 0 and -inf, the others are untouched by them."""
    c = Case([0, max(1, n - 2), 70], [n, n, n], G=G, seed=n, pad=2)
    out, l = c.check()
    assert (out[:n] == 0).all() and torch.isneginf(l[:n]).all()
    c.check(causal=False)


@pytest.mark.parametrize("n,G", [(1, 2), (4, 4), (20, 5)])
def test_not_causal(n, G):
    Case([90, 5], [n, n], G=G, seed=3).check(causal=False)


def test_sequences_without_rows_and_padded_batch():
    Case([50, 60, 0, 70], [2, 0, 0, 3], pad=5, seed=4).check()
    Case([50, 60, 20, 70], [20, 0, 1, 33], pad=5, seed=5).check()


@pytest.mark.parametrize("n,G", [(1, 4), (9, 4)])
def test_scale_signs_and_peaks(n, G):
    c = Case([120, 33], [n, n], G=G, seed=6)
    for scale in (0.0, -0.2, 1.5):
        c.check(scale=scale)


def test_values_of_very_different_size():
    """Tokens whose values differ by 2^20 from one to the next (the weights' factor follows the largest seen)."""
    c = Case([96, 64], [1, 1], seed=7, P=16)
    rng = np.random.default_rng(8)
    kv = torch.tensor(rng.standard_normal((2, 160, 2, 128)), dtype=torch.float32)
    kv[1] *= torch.tensor(2.0 ** rng.integers(-10, 11, 160))[:, None, None].float()
    kv = kv.bfloat16().cuda()
    q.mla_qcache_kv4_append(c.cfg, kv[0], kv[1], offsets([96, 64]), ints([0, 0]), 96, ints(c.table), c.pool, c.err)
    c.check()
    c.check(scale=1.0)


@pytest.mark.parametrize("n", [1, 12])
def test_long_sequences_in_many_parts_are_repeatable(n):
    """One item over many CTAs: joined in a fixed order, so two calls agree bit for bit, whatever ran in between."""
    c = Case([9001, 4000], [n, n], Hkv=1, G=8, P=64, seed=9)
    ws = c.workspace()
    a = c.check(ws=ws)
    Case([5, 5], [1, 1], Hkv=1, G=8, P=64, seed=1).run(ws=ws)
    b = c.run(ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not ws[:8192].any()  # the counters are zero between calls


def test_one_workspace_for_calls_of_other_sizes():
    cases = [Case([700, 90], [1, 1], Hkv=1, G=4, seed=1), Case([700, 90], [4, 4], Hkv=1, G=4, seed=2),
             Case([700, 900], [30, 2], Hkv=1, G=4, seed=3), Case([700, 900], [90, 2], Hkv=1, G=4, seed=4)]
    ws = torch.zeros(max(c.workspace().numel() for c in cases), dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        c.check(ws=ws, lse=max(c.new) < 30)


@pytest.mark.parametrize("n", [1, 20])
def test_many_short_sequences(n):
    """More sequences than a warp's lanes hold in registers, and more items than CTAs."""
    rng = np.random.default_rng(n)
    B = 700 if n == 1 else 40
    lens = [int(x) for x in rng.integers(n, n + 60, B)]
    Case(lens, [n] * B, Hkv=2, G=2, D=64, P=16, seed=n).check()


def test_sequence_lengths_of_very_different_size():
    Case([3000, 1, 17, 2000, 64, 1, 900, 33], [1] * 8, Hkv=2, G=4, P=32, seed=5).check()
    Case([3000, 1, 17, 2000], [6, 1, 6, 2], Hkv=2, G=4, P=32, seed=6).check()


def test_pages_beyond_four_gigabytes():
    """Page ids whose byte offset passes 32 bits."""
    c = Case([40, 100], [1, 1], Hkv=8, G=4, P=128, seed=2)
    far = (1 << 32) // q.kv4_page_bytes(c.cfg) + 5
    pool = torch.empty((far + 4, c.pool.shape[1]), dtype=torch.uint8, device="cuda")
    ids = [far, far + 3]
    for b in range(2):
        pool[ids[b]] = c.pool[int(c.table[b, 0])]
    a = c.run()
    small, c.pool, c.table = (c.pool, c.table), pool, np.array([[ids[0], 0], [ids[1], 0]], np.int32)
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and int(c.err) == 0
    # and the append to them
    kv = torch.randn(2, 1, 8, 128, device="cuda").bfloat16()
    for pl, tb in ((pool, c.table), small):
        q.mla_qcache_kv4_append(c.cfg, kv[0], kv[1], ints([0, 1, 1]), ints([40, 100]), 1, ints(tb), pl, c.err)
    assert torch.equal(pool[ids[0]], small[0][int(small[1][0, 0])]) and int(c.err) == 0


@pytest.mark.parametrize("n,G", [(1, 4), (2, 8), (20, 4)])
def test_bad_page_leaves_its_tokens_out(n, G):
    c = Case([64], [n], Hkv=1, G=G, P=16, seed=3)
    good = c.table.copy()
    c.table[0, 1] = c.n_pages
    out, l = c.run(causal=False)
    assert int(c.err) == q.DEV_BAD_PAGE and torch.isfinite(out).all()
    c.err.zero_()
    c.table = good
    pool = c.pool.cpu().numpy()
    k, v, vs, most = ref.read_sequence(pool, good[0], 64, 1, 128, 128, 16)
    ok = np.ones((n, 64), bool)
    ok[:, 16:32] = False
    want, _, bound = ref.attention(c.q.double().cpu().numpy(), k, v, vs, most, 1 / math.sqrt(128), ok, c.t, n * G > 16)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("n,G", [(1, 4), (20, 4)])
def test_lengths_and_rows_out_of_range(n, G):
    c = Case([64, 40], [n, n], Hkv=1, G=G, P=16, seed=3)
    keep = list(c.lens)
    c.lens = [keep[0], 16 * c.table.shape[1] + 1]
    out, l = c.run()
    assert int(c.err) == q.DEV_SEQ_OVERFLOW and (out[n:] == 0).all() and torch.isneginf(l[n:]).all()
    c.err.zero_()
    c.lens, c.new = keep, [n, n]
    out = torch.full_like(out, 7.0)
    q.mla_qcache_kv4_attn(c.cfg, c.q, ints(c.table), ints(c.lens), c.pool, 0.1, out, c.workspace(), c.err,
                          cu_q=ints([0, n, 2 * n + 50]), max_q=n)
    assert int(c.err) == q.DEV_ROWS and (out[n:] == 7).all() and (out[:n] != 7).any()


def test_strided_queries_and_infinities_in_other_rows():
    """Queries as a view of a projection's output; a row of infinities or NaN does not reach the other rows."""
    for n, G in ((1, 4), (12, 4)):
        c = Case([80, 50], [n, n], Hkv=2, G=G, seed=4)
        wide = torch.full((2 * n, c.Hq + 4, 128), float("nan"), dtype=c.t, device="cuda")
        wide[:, :c.Hq] = c.q
        a, _ = c.check()
        b, _ = c.run(qq=wide[:, :c.Hq])
        assert torch.equal(a, b)
        bad = c.q.clone()
        bad[0, 0] = float("inf")
        bad[n, 3] = float("nan")
        d, _ = c.run(qq=bad)
        keep = torch.ones(2 * n, c.Hq, dtype=torch.bool)
        keep[0, 0] = keep[n, 3] = False
        assert torch.equal(a[keep], d[keep])


def test_refusals_on_the_device():
    c = Case([40], [2], G=2)
    with pytest.raises(q.QCacheError, match="workspace"):
        c.run(ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        c.run(out=torch.empty(2, 4, 64, dtype=c.t, device="cuda"))
    with pytest.raises(q.QCacheError, match="out"):
        c.run(out=torch.empty(2, 4, 128, device="cuda"))
    with pytest.raises(q.QCacheError, match="contiguous"):
        c.run(out=torch.empty(4, 2, 128, dtype=c.t, device="cuda").transpose(0, 1))
    with pytest.raises(q.QCacheError, match="float16"):
        c.run(qq=c.q.float())
    with pytest.raises(ValueError, match="pool"):
        c.pool, keep = c.pool[:, :-16].contiguous(), c.pool
        c.run()
    c.pool = keep
    with pytest.raises(q.QCacheError):  # a window without a causal mask
        c.run(causal=False, window=3)
    with pytest.raises(q.QCacheError, match="cpu"):
        q.mla_qcache_kv4_attn(c.cfg, c.q, ints(c.table).cpu(), ints(c.lens), c.pool, 0.1, c.q, c.workspace(), c.err, cu_q=offsets([2]), max_q=2)


# ---------------------------------------------------------------- as they are used
def test_prompt_then_decode_steps_agree_with_dense_attention():
    """A decoder's life: a prompt is appended and attended to, in two chunks, then single tokens and drafted ones.
    Each step agrees with dense attention in 64 bits over the values that the appends report."""
    rng = np.random.default_rng(0)
    B, Hkv, G, D, P, group = 3, 2, 4, 128, 32, 64
    cfg = q.make_kv4_config(Hkv, D, group=group, page_size=P)
    pages = 8
    table = ints(rng.permutation(B * pages).reshape(B, pages))
    pool = torch.zeros((B * pages, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    cos, sin = (torch.tensor(x).cuda() for x in tables(P * pages, D))
    lens, nxt, err = ints([0] * B), ints([0] * B), error_word()
    ws = torch.zeros(max(q.kv4_workspace_bytes(cfg, B, Hkv * G, m, pages) for m in (1, 4, 50, 60)), dtype=torch.uint8, device="cuda")
    held = [[], [], []]
    for new in ([40, 7, 50], [33, 60, 0], [1, 1, 1], [1, 1, 1], [4, 3, 4], [1, 0, 1]):
        rows = sum(new)
        qkv = torch.tensor(rng.standard_normal((rows, (G + 2) * Hkv, D)), dtype=torch.float32).bfloat16().cuda()
        qr = torch.empty(rows, G * Hkv, D, dtype=torch.bfloat16, device="cuda")
        kd, vd = (torch.empty(rows, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cu = offsets(new)
        q.mla_qcache_kv4_append(cfg, qkv[:, G * Hkv:(G + 1) * Hkv], qkv[:, (G + 1) * Hkv:], cu, lens, max(new), table, pool, err,
                                cos=cos, sin=sin, q=qkv[:, :G * Hkv], q_out=qr, k_deq=kd, v_deq=vd, seq_lens_next=nxt)
        lens, nxt = nxt, lens
        out = torch.empty_like(qr)
        q.mla_qcache_kv4_attn(cfg, qr, table, lens, pool, D ** -0.5, out, ws, err, cu_q=cu, max_q=max(new))
        torch.cuda.synchronize()
        r = 0
        for b, n in enumerate(new):
            held[b].append((kd[r:r + n].double().cpu(), vd[r:r + n].double().cpu()))
            if n:
                k, v = (torch.cat([x[i] for x in held[b]]) for i in range(2))
                T = k.shape[0]
                assert T == int(lens[b])
                ok = torch.tensor(ref.seen(T, n, True, 0))
                for h in range(G * Hkv):
                    s = qr[r:r + n, h].double().cpu() @ k[:, h // G].T * D ** -0.5
                    want = s.masked_fill(~ok, -math.inf).softmax(-1) @ v[:, h // G]
                    # the reported values are rounded to BF16 (2^-9 of a value): once in the scores, once in the result
                    mag = (qr[r:r + n, h].double().cpu().abs() @ k[:, h // G].abs().T * D ** -0.5).amax(-1, keepdim=True)
                    tol = (2 * 2.0 ** -9 * mag + 3 * 2.0 ** -8) * v[:, h // G].abs().amax()
                    assert ((out[r:r + n, h].double().cpu() - want).abs() <= tol).all()
            r += n
    assert int(err) == 0


def test_captured_steps_replay_with_new_inputs():
    """A decode step (append with rotation, attention) captured once and replayed: lengths, tokens and queries change
    in place. Two graphs with workspaces of their own run on two streams at once."""
    rng = np.random.default_rng(1)
    graphs = []
    for seed in (1, 2):
        c = Case([70, 33], [1, 1], Hkv=2, G=4, P=16, seed=seed, spare=3)
        cos, sin = (torch.tensor(x).cuda() for x in tables(200, 128))
        st = dict(c=c, lens=ints(c.lens), nxt=ints([0, 0]), cu=ints([0, 1, 2]), table=ints(c.table), ws=c.workspace(), cos=cos, sin=sin,
                  kv=torch.empty(2, 2, 2, 128, dtype=c.t, device="cuda"), qr=torch.empty_like(c.q), out=torch.empty_like(c.q),
                  lse=torch.empty(2, c.Hq, device="cuda"))

        def step(st=st, c=c):
            q.mla_qcache_kv4_append(c.cfg, st["kv"][0], st["kv"][1], st["cu"], st["lens"], 1, st["table"], c.pool, c.err, cos=st["cos"],
                                    sin=st["sin"], q=c.q, q_out=st["qr"], seq_lens_next=st["nxt"])
            q.mla_qcache_kv4_attn(c.cfg, st["qr"], st["table"], st["nxt"], c.pool, 0.09, st["out"], st["ws"], c.err, lse=st["lse"])
            st["lens"].copy_(st["nxt"])
        keep = st["lens"].clone()
        step()
        st["lens"].copy_(keep)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, st, torch.cuda.Stream()))
    for i in range(20):
        torch.cuda.synchronize()
        for _, st, _ in graphs:
            st["kv"].copy_(torch.tensor(rng.standard_normal(st["kv"].shape), dtype=torch.float32).to(st["c"].t))
            st["c"].q.copy_(torch.tensor(rng.standard_normal(st["c"].q.shape), dtype=torch.float32).to(st["c"].t))
        torch.cuda.synchronize()
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, st, _ in graphs:
            c = st["c"]
            c.lens = st["lens"].tolist()
            assert c.lens == [71 + i, 34 + i] and int(c.err) == 0
            qq, c.q = c.q, st["qr"]
            if i % 7 == 6:
                a, l = c.check(scale=0.09, one=True)
                assert torch.equal(a, st["out"]) and torch.equal(l, st["lse"])
            c.q = qq


def test_a_stream_of_ones_own():
    c = Case([900, 300], [1, 1], Hkv=1, G=8, P=64, seed=5)
    a, _ = c.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = c.run(stream=s)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("G,n", [(4, 6), (4, 11), (8, 12), (4, 60)])
def test_captured_many_rows_replay_over_other_lengths(G, n):
    """The calls of the many-row kernels captured once, replayed while the sequences grow, shrink and empty."""
    c = Case([40, 4500, 9], [n, n, n], Hkv=1, G=G, P=32, seed=n, spare=2)
    full, lens, table, cu = list(c.lens), ints(c.lens), ints(c.table), offsets(c.new)
    out, ws = torch.empty_like(c.q), c.workspace()
    lse = torch.empty(sum(c.new), c.Hq, device="cuda")

    def call():
        q.mla_qcache_kv4_attn(c.cfg, c.q, table, lens, c.pool, 0.1, out, ws, c.err, cu_q=cu, max_q=n, lse=lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lengths in (full, [min(n, full[0]), 130, 0], [1, 4097, 9], [0, 0, 0], [33, 2047, 1], full):
        lens.copy_(ints(lengths))
        g.replay()
        torch.cuda.synchronize()
        c.lens = lengths
        a, l = c.check(scale=0.1)
        assert torch.equal(a, out) and torch.equal(l, lse)


def test_workspace_serves_every_call_up_to_its_sizes():
    """One workspace of max_q rows and the table's pages for calls of fewer rows, in any order (the counters stay zero)."""
    for Hkv, G in ((1, 4), (13, 4), (1, 300)):
        c = Case([5000, 70], [700 if G == 4 else 3, 1], Hkv=Hkv, G=G, D=64, P=256, seed=G)
        ws, most = c.workspace(700), c.new[0]
        for n in (most, 1, min(most, 9), min(most, 20), min(most, 33), min(most, 65), 2):
            c.new = [n, 1]
            c.run(ws=ws, max_q=700, lse=bool(n & 1), qq=c.q[:n + 1])
            torch.cuda.synchronize()
            assert int(c.err) == 0 and not ws[:8192].any()


def test_cache_object_prompt_then_steps():
    """KV4Cache: a prompt with rotation, then decode steps, against dense attention over what the cache holds."""
    rng, D, Hkv, G = np.random.default_rng(2), 128, 2, 4
    cfg = q.make_kv4_config(Hkv, D, group=64, page_size=32)
    cache = q.KV4Cache(cfg, 2, 6)
    cos, sin = (torch.tensor(x).cuda() for x in tables(200, D))
    for new in ([100, 37], [1, 1], [1, 1], [4, 2]):
        rows = sum(new)
        qkv = torch.tensor(rng.standard_normal((rows, Hkv * (G + 2), D)), dtype=torch.float32).bfloat16().cuda()
        qr = torch.empty(rows, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
        cache.append(qkv[:, Hkv * G:-Hkv], qkv[:, -Hkv:], offsets(new), max(new), cos=cos, sin=sin, q=qkv[:, :Hkv * G], q_out=qr)
        lse = torch.empty(rows, Hkv * G, device="cuda")
        out = cache.attend(qr, D ** -0.5, cu_q=offsets(new), max_q=max(new), lse=lse)
        torch.cuda.synchronize()
        assert cache.error_bits() == 0
        pool, r = cache.pool.cpu().numpy(), 0
        for b, n in enumerate(new):
            T = int(cache.seq_lens[b])
            k, v, vs, most = ref.read_sequence(pool, cache.page_table[b].cpu().numpy(), T, Hkv, D, 64, 32)
            qq = qr[r:r + n].double().cpu().numpy()
            want, wl, bound = ref.attention(qq, k, v, vs, most, D ** -0.5, ref.seen(T, n, True, 0), torch.bfloat16, max(new) * G > 16)
            assert (np.abs(out[r:r + n].double().cpu().numpy() - want) <= bound).all()
            r += n
    assert cache.seq_lens.tolist() == [106, 41]

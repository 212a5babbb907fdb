"""Attention of trees of drafted tokens over the grouped-query cache in 4 bits, the append of their nodes, their masks and what stays of
them, on the GPU against the plain statements (kv4_ref, tree_ref), within the bounds of kv4_paths."""
import math

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import kv4_paths, kv4_ref as ref, tree_ref as tr
from tests.test_gpu_kv4 import Case, TYPES, error_word, ints, offsets, tables

pytestmark = pytest.mark.gpu


WIDE = False


@pytest.fixture(params=["short", "wide"], autouse=True)
def room(request):
    """Tables as long as the sequences, or with room for 2^20 tokens: which kernel takes a call goes by it."""
    global WIDE
    WIDE = request.param == "wide"


def stays_few(c, rows):
    """33 to 128 rows whose blocks of eight are few and short stay with the kernel for few rows."""
    items = -(-rows // 8) * len(c.lens) * c.Hkv
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rows <= 128 and items <= 2 * sms and items * c.table.shape[1] * c.P * c.D <= 9 << 22


class Tree(Case):
    """lens: tokens with the tree, sizes: nodes of each tree, new: rows of queries, the tree's newest nodes."""

    def __init__(self, lens, sizes, new=None, words=None, chain=False, **kw):
        super().__init__(lens, sizes if new is None else new, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + 1000)
        self.base = [T - n for T, n in zip(lens, sizes)]
        if WIDE:
            self.table = np.ascontiguousarray(np.concatenate([self.table, np.full((len(lens), 2 ** 20 // self.P), 10 ** 6, np.int32)], 1))
        self.words = words or max(1, -(-max(sizes) // 64))
        self.masks = []
        for n, rows in zip(sizes, self.new):
            ms = tr.masks([i - 1 for i in range(n)] if chain else tr.random_parents(rng, n)) if n else []
            self.masks.append(ms[n - rows:])

    def run(self, scale=None, window=0, lse=True, ws=None, max_q=None, qq=None, base=..., masks=None, lens=None, table=None, stream=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        rows = sum(self.new) + self.pad
        out = torch.full((rows, self.Hq, self.D), 7.0, dtype=self.t, device="cuda")
        l = torch.full((rows, self.Hq), 7.0, device="cuda") if lse else None
        max_q = max_q or max(1, max(self.new))
        flat = [m for ms in (masks or self.masks) for m in ms] + [(1 << 64) - 1] * self.pad
        q.mla_qcache_kv4_attn_tree(self.cfg, self.q if qq is None else qq, tr.mask_tensor(flat, self.words), offsets(self.new), max_q,
                                   ints(self.table if table is None else table), ints(lens or self.lens), self.pool, scale, out,
                                   self.workspace(max_q) if ws is None else ws, self.err,
                                   tree_base=ints(self.base) if base is ... else base, lse=l, window=window, stream=stream)
        return out, l

    def compare(self, out, l, scale=None, window=0, hide=None, masks=None, max_q=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        pool, r = self.pool.cpu().numpy(), 0
        rows = (max_q or max(1, max(self.new))) * (self.Hq // self.Hkv)
        way = "few" if stays_few(self, rows) else kv4_paths.path(rows, self.D, l is not None)
        for b, (T, n, base) in enumerate(zip(self.lens, self.new, self.base)):
            k, v, vs, most = ref.read_sequence(pool, self.table[b], T, self.Hkv, self.D, self.group, self.P)
            ok = tr.seen(T, base, (masks or self.masks)[b], self.words, window)
            if hide is not None:
                ok &= ~hide[b][None, :T]
            qq = self.q[r:r + n].double().cpu().numpy()
            want, wl, bound = kv4_paths.attention(qq, k, v, vs, most, scale, ok, self.t, way)
            got = out[r:r + n].double().cpu().numpy()
            assert np.isfinite(got).all()
            off = np.abs(got - want)
            assert (off <= bound).all(), f"{way}, sequence {b}: {(off - bound).max():.3e} beyond the bound"
            assert not got[~ok.any(1)].any()  # rows that see nothing
            if l is not None:
                gl = l[r:r + n].double().cpu().numpy()
                fin = np.isfinite(wl)
                assert np.array_equal(np.isneginf(gl), ~fin)
                far = np.abs(gl[fin] - wl[fin])
                assert (far <= (ref.lse_bound(qq, k, scale, ok) + kv4_paths.query_error(qq, k, scale, ok))[fin]).all(), far.max()
            r += n
        if self.pad:
            assert (out[r:] == 7).all() and (l is None or (l[r:] == 7).all())

    def check(self, window=0, lse=True, **kw):
        out, l = self.run(window=window, lse=lse, **kw)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        self.compare(out, l, window=window, max_q=kw.get("max_q"), masks=kw.get("masks"))
        return out, l


# few rows: up to 32 of a kv head; one tile of queries up to 128 (64: held twice), two above
@pytest.mark.parametrize("D,group,P,Hkv,G,dtype,size", [
    (128, 128, 64, 2, 4, "bf16", 8), (128, 64, 16, 1, 1, "fp16", 7), (64, 64, 16, 2, 7, "fp16", 4), (64, 32, 128, 1, 2, "bf16", 16),
    (128, 32, 32, 2, 8, "bf16", 4), (128, 128, 64, 2, 4, "fp16", 16), (64, 64, 32, 2, 7, "bf16", 9), (128, 64, 16, 1, 5, "bf16", 20),
    (64, 32, 16, 1, 4, "fp16", 30), (128, 32, 256, 1, 8, "bf16", 26), (128, 128, 32, 1, 16, "fp16", 33), (64, 64, 64, 1, 16, "bf16", 20)])
@pytest.mark.parametrize("lse", [True, False])
def test_layouts_and_kernels(D, group, P, Hkv, G, dtype, size, lse):
    Tree([300, size, size + 1, 131 + size], [size, size, max(1, size - 3), 1], Hkv=Hkv, G=G, D=D, group=group, P=P, dtype=dtype,
         seed=D + size, pad=2).check(lse=lse)


@pytest.mark.parametrize("G,n", [(1, 9), (4, 3), (4, 4), (7, 2), (7, 3), (8, 3), (5, 5), (8, 4), (32, 1)])
@pytest.mark.parametrize("D,group,P,dtype", [(128, 64, 64, "fp16"), (64, 64, 16, "bf16"), (128, 128, 128, "bf16"), (128, 32, 32, "bf16")])
def test_up_to_32_rows(G, n, D, group, P, dtype):
    """Blocks of 8 or 16 rows, by the table's room: both hold their bounds, for nodes and for last positions."""
    args = dict(Hkv=2, G=G, D=D, group=group, P=P, dtype=dtype, seed=G + n)
    c = Tree([700, 40 + n, n, 0], [n, n, n, 0], **args)
    plain = Case([700, 40 + n, n, 0], [n, n, n, 0], **args)
    plain.table = np.ascontiguousarray(np.concatenate([plain.table, c.table[:, plain.table.shape[1]:]], 1))
    for x in (c, plain):
        x.check()
        x.check(window=33)


@pytest.mark.parametrize("size", [1, 2, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 256])
def test_sizes_of_trees(size):
    Tree([size + 37, size], [size, size], Hkv=1, G=2, D=64, P=16, seed=size).check()


@pytest.mark.parametrize("base", [0, 1, 15, 16, 31, 32, 33, 95, 96, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("G,size", [(4, 7), (8, 12), (8, 24)])
def test_places_of_the_tree_in_tiles_and_pages(base, G, size):
    Tree([base + size], [size], Hkv=1, G=G, P=32, seed=base).check()


@pytest.mark.parametrize("G,size,new", [(7, 24, 4), (4, 40, 8), (8, 70, 5), (2, 130, 30), (8, 256, 40), (1, 9, 0)])
def test_the_newest_nodes_alone(G, size, new):
    Tree([500, 90 + size, size], [size, size, size], new=[new, min(1, new), new], Hkv=2, G=G, D=64, P=16, seed=size).check()


@pytest.mark.parametrize("window", [1, 2, 5, 16, 31, 33, 64, 100, 129, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("G,size", [(4, 8), (8, 20), (8, 40)])
def test_windows(window, G, size):
    """A node deep in the tree sees less of the tokens before it; pages that nobody sees are not read."""
    c = Tree([301, 70 + size, size + 3], [size, size, size], Hkv=1, G=G, D=64, P=16, seed=window % 97)
    table = c.table.copy()
    for b, base in enumerate(c.base):  # ids of pages behind the window may be anything
        table[b, :max(0, base - window) // c.P] = 10 ** 6
    out, l = c.run(window=window, table=table)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.compare(out, l, window=window)


@pytest.mark.parametrize("G,size", [(4, 8), (8, 24)])
@pytest.mark.parametrize("window", [0, 20])
def test_masks_of_any_bits(G, size, window):
    """Rows that do not see themselves, that see nothing, or whose masks name nodes that are not there."""
    c = Tree([180, size, size + 2], [size, size, size], words=4, Hkv=1, G=G, P=16, seed=size)
    rng = np.random.default_rng(7)
    some = [[int.from_bytes(rng.bytes(32), "little") & int.from_bytes(rng.bytes(32), "little") for _ in range(size)] for _ in range(3)]
    some[0][0] = some[1][0] = some[2][1] = 0
    some[0][1] = (1 << 256) - 1
    c.check(masks=some, window=window)


def test_nothing_before_the_tree_and_empty_masks():
    c = Tree([6, 6], [6, 6], Hkv=1, G=4, P=16)
    c.check(masks=[[0] * 6, [1 << i for i in range(6)]])


@pytest.mark.parametrize("G,size", [(4, 8), (8, 30)])
def test_chains_are_causal_rows(G, size):
    """A chain's masks are the causal mask, and the base need not be given where the rows are the whole tree."""
    c = Tree([400, 33 + size], [size, size], chain=True, Hkv=2, G=G, P=64, seed=4)
    out, l = c.check()
    same, sl = c.run(base=None)
    rows, rl = Case.run(c)
    torch.cuda.synchronize()
    assert torch.equal(same, out) and torch.equal(sl, l)
    # both lie within the bound around the same values
    tol = 2 * 2.0 ** -8 * rows.float().abs() + 1e-2
    assert ((rows.float() - out.float()).abs() <= tol).all() and (rl - l).abs().max() < 1e-3


def test_long_sequences_in_parts():
    """Items cut over the CTAs and joined, in both kernels and on the line."""
    for lens, sizes, G in (([9000, 300, 5000], [7, 8, 3], 4), ([9000, 2100, 40], [26, 20, 26], 8), ([5000] * 20, [12] * 20, 4)):
        Tree(lens, sizes, Hkv=2, G=G, P=64, seed=len(lens)).check()


@pytest.mark.parametrize("D,group,G,size,dtype", [(64, 32, 7, 9, "fp16"), (64, 64, 8, 16, "bf16"), (64, 64, 16, 20, "fp16"), (128, 64, 8, 14, "fp16")])
@pytest.mark.parametrize("lse", [True, False])
def test_parts_of_every_form_are_joined(D, group, G, size, dtype, lse):
    """64, 128 and 256 rows to an item, cut over the CTAs."""
    Tree([6000, 2500, size, 4001], [size, size, size, 3], Hkv=1, G=G, D=D, group=group, P=64, dtype=dtype, seed=size).check(lse=lse)


def test_more_sequences_than_a_warp_or_a_block_looks_at():
    """40 pairs on the line are shared out by the block; 600 sequences are not ordered by length; 70 are."""
    Tree([2600] + [int(x) for x in np.random.default_rng(0).integers(12, 400, 39)], [12] * 40, Hkv=1, G=4, P=64, seed=1).check()
    for B in (70, 600):
        Tree([int(x) for x in np.random.default_rng(B).integers(9, 200, B)], [9] * B, Hkv=1, G=4, D=64, P=16, seed=B).check()


def test_strided_queries_masks_of_one_dimension_and_other_streams():
    c = Tree([77, 150], [6, 7], Hkv=2, G=4, P=16)
    out, l = c.check()
    wide = torch.full((sum(c.new), c.Hq + 3, c.D + 8), float("nan"), dtype=c.t, device="cuda")
    wide[:, 2:2 + c.Hq, :c.D] = c.q
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        o2, l2 = c.run(qq=wide[:, 2:2 + c.Hq, :c.D], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, l)
    flat = tr.mask_tensor([m for ms in c.masks for m in ms], 1)[:, 0].contiguous()
    o3 = torch.zeros_like(out)
    q.mla_qcache_kv4_attn_tree(c.cfg, c.q, flat, offsets(c.new), 7, ints(c.table), ints(c.lens), c.pool, c.D ** -0.5, o3, c.workspace(),
                               c.err, tree_base=ints(c.base))
    torch.cuda.synchronize()
    assert (o3.float() - out.float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()


@pytest.mark.parametrize("G,size", [(4, 6), (8, 20)])
def test_what_is_reported(G, size):
    c = Tree([120, 64 + size], [size, size], Hkv=1, G=G, P=16)
    want, wl = c.check()
    n = c.new[0]

    def word(**kw):
        c.err.zero_()
        out, l = c.run(**kw)
        torch.cuda.synchronize()
        return int(c.err), out, l
    for base in (-1, 121):  # outside [0, T]: the sequence is empty, the other as it was
        e, out, l = word(base=ints([base, c.base[1]]))
        assert e == q.DEV_SEQ_OVERFLOW and (out[:n] == 0).all() and torch.isneginf(l[:n]).all()
        assert torch.equal(out[n:], want[n:])
    e, out, _ = word(lens=[c.table.shape[1] * c.P + 1, c.lens[1]])
    assert e & q.DEV_SEQ_OVERFLOW and (out[:n] == 0).all() and torch.equal(out[n:], want[n:])
    e, out, l = word(max_q=size, base=None, lens=[size - 1, c.lens[1]])  # more rows than tokens
    assert e == q.DEV_SEQ_OVERFLOW and (out[:n] == 0).all()
    for at in (1, 7):  # a page before the tree, and the tree's own
        table = c.table.copy()
        table[0, at] = c.n_pages
        e, out, l = word(table=table)
        assert e == q.DEV_BAD_PAGE
        hide = [np.zeros(T, bool) for T in c.lens]
        hide[0][16 * at:16 * at + 16] = True
        c.compare(out, l, hide=hide)


@pytest.mark.parametrize("G,size", [(4, 8), (8, 16)])
def test_captured_calls_follow_lengths_and_masks(G, size):
    c = Tree([200, 90], [size, size], Hkv=1, G=G, P=16, spare=3)
    lens, base = ints(c.lens), ints(c.base)
    mask, cu = tr.mask_tensor([m for ms in c.masks for m in ms], 1), offsets(c.new)
    out, l = torch.zeros(2 * size, c.Hq, c.D, dtype=c.t, device="cuda"), torch.zeros(2 * size, c.Hq, device="cuda")
    ws, table = c.workspace(), ints(c.table)
    call = lambda: q.mla_qcache_kv4_attn_tree(c.cfg, c.q, mask, cu, size, table, lens, c.pool, c.D ** -0.5, out, ws, c.err,  # noqa: E731
                                              tree_base=base, lse=l)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    rng = np.random.default_rng(5)
    for back in (0, 3, 70):
        c.lens, c.base = [200 - back, 90 - back], [200 - back - size, 90 - back - size]
        c.masks = [tr.masks(tr.random_parents(rng, size)) for _ in range(2)]
        lens.copy_(ints(c.lens)), base.copy_(ints(c.base)), mask.copy_(tr.mask_tensor([m for ms in c.masks for m in ms], 1))
        g.replay()
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.compare(out, l)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("D,rot,interleaved,dtype,words", [(128, 128, False, "bf16", 1), (64, 32, True, "fp16", 2), (128, 64, False, "fp16", 4)])
@pytest.mark.parametrize("late", [False, True])
def test_append_of_a_tree_turns_siblings_alike(D, rot, interleaved, dtype, words, late):
    """Rows go behind the sequence's tokens and are rotated by their depth; `late`: a level of trees that began three tokens earlier."""
    rng = np.random.default_rng(D + rot)
    t, P, Hkv, Hq = TYPES[dtype], 16, 2, 4
    cfg = q.make_kv4_config(Hkv, D, group=32, page_size=P)
    sizes, lens = [9, 0, 14], [13, 5, 0 if not late else 3]
    base = [x - 3 for x in lens] if late else lens
    ms = [tr.masks(tr.random_parents(rng, n + 3 * late))[3 * late:] for n in sizes]
    rows = sum(sizes)
    x = torch.tensor(rng.standard_normal((rows, Hq + 2 * Hkv, D)), dtype=torch.float32).to(t).cuda()
    cos, sin = tables(40, rot)
    table = rng.permutation(12).astype(np.int32).reshape(3, 4)
    pool = torch.randint(0, 256, (12, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    want, err, nxt = pool.cpu().numpy().copy(), error_word(), ints([-1] * 3)
    q_out = torch.zeros(rows, Hq, D, dtype=t, device="cuda")
    q.mla_qcache_kv4_append(cfg, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], offsets(sizes), ints(lens), max(sizes), ints(table), pool, err,
                            cos=torch.tensor(cos).cuda(), sin=torch.tensor(sin).cuda(), interleaved=interleaved, q=x[:, :Hq], q_out=q_out,
                            seq_lens_next=nxt, tree_mask=tr.mask_tensor([m for s in ms for m in s], words),
                            tree_base=ints(base) if late else None)
    torch.cuda.synchronize()
    assert int(err) == 0 and nxt.tolist() == [a + n for a, n in zip(lens, sizes)]
    pos = np.array([b + bin(m).count("1") - 1 for b, s in zip(base, ms) for m in s])
    f = x.float().cpu().numpy()
    qk = ref.rotate32(f[:, :Hq + Hkv], cos[pos], sin[pos], interleaved)
    kq, vq = ref.quantize(qk[:, Hq:].astype(np.float64), 32), ref.quantize(f[:, Hq + Hkv:].astype(np.float64), 32)
    r = 0
    for b, (T, n) in enumerate(zip(lens, sizes)):
        for i in range(n):
            for h in range(Hkv):
                ref.put_token(want, table[b, (T + i) // P], (T + i) % P, h, D, 32, P, [a[r, h] for a in kq], [a[r, h] for a in vq])
            r += 1
    assert np.array_equal(pool.cpu().numpy(), want)
    assert torch.equal(q_out.cpu(), torch.tensor(qk[:, :Hq]).to(t))


def test_append_of_a_tree_reports_positions_without_angles():
    cfg = q.make_kv4_config(1, 64, page_size=16)
    k = torch.randn(3, 1, 64, device="cuda").bfloat16()
    ang = torch.ones(6, 32, device="cuda")

    def run(ms, base=None, lens=4, rotated=True):
        pool, err = torch.zeros((2, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda"), error_word()
        q.mla_qcache_kv4_append(cfg, k, k, ints([0, 3]), ints([lens]), 3, ints([[0, 1]]), pool, err, cos=ang if rotated else None,
                                sin=ang if rotated else None, tree_mask=tr.mask_tensor(ms, 1), tree_base=base)
        codes = pool[0, :16 * 32].view(16, 32)
        return int(err), [t for t in range(16) if bool((codes[t] != 0).any())]
    assert run([1, 3, 5]) == (0, [4, 5, 6])
    assert run([1, 3, 7]) == (q.DEV_SEQ_OVERFLOW, [4, 5])             # position 6 of a table of six
    assert run([1, 3, 7], rotated=False) == (0, [4, 5, 6])
    assert run([0, 1, 1], lens=0) == (q.DEV_SEQ_OVERFLOW, [1, 2])     # position -1
    assert run([1, 3, 7], base=ints([2])) == (0, [4, 5, 6])


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("words", [1, 2, 3, 4])
def test_masks_from_parents(words):
    rng = np.random.default_rng(words)
    most = 64 * words
    sizes = [1, most, 0, 33, most - 1]
    ps = [tr.random_parents(rng, n) if n else [] for n in sizes]
    ps[3] = [-1] * 33  # roots alone
    ps[4] = [i - 1 for i in range(sizes[4])]
    rows, pad = sum(sizes), 2
    mask = torch.full((rows + pad, words), 7, dtype=torch.int64, device="cuda")
    err = error_word()
    q.mla_qcache_tree_mask(ints([x for p in ps for x in p] + [0] * pad), offsets(sizes), most, mask, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and (mask[rows:] == 7).all()
    assert torch.equal(mask[:rows], tr.mask_tensor([m for p in ps for m in (tr.masks(p) if p else [])], words))


def test_masks_from_bad_parents():
    err, mask = error_word(), torch.full((7,), 7, dtype=torch.int64, device="cuda")
    q.mla_qcache_tree_mask(ints([-1, 0, 2, -5, 1, 0, 0]), ints([0, 5, 7]), 5, mask, err)
    assert int(err) == q.DEV_ROWS and mask.tolist() == [1, 3, 4, 8, 16 + 3, 1, 3]
    err.zero_(), mask.fill_(7)
    q.mla_qcache_tree_mask(ints([-1, 0, 1, -1, 0, 0, 0]), ints([0, 3, 7]), 3, mask, err)
    assert int(err) == q.DEV_ROWS and mask.tolist() == [1, 3, 7, 7, 7, 7, 7]


# ---------------------------------------------------------------- keep
@pytest.mark.parametrize("D,group,P,Hkv", [(128, 128, 64, 2), (128, 64, 16, 3), (128, 32, 128, 1), (64, 64, 16, 2), (64, 32, 256, 5)])
@pytest.mark.parametrize("most", [1, 2, 9, 64, 255, 256])
def test_keep_moves_tokens_past_one_another(D, group, P, Hkv, most):
    rng = np.random.default_rng(D + P + most)
    cfg = q.make_kv4_config(Hkv, D, group=group, page_size=P)
    base = [0, P - 1, 3 * P + 5, 17, 2]
    far = [256, 256, most, 300, 400]  # nodes lie within
    count = [most, most, most, 0, int(rng.integers(1, most + 1))]
    pages = -(-(max(base) + 400) // P)
    table = rng.permutation(5 * pages).astype(np.int32).reshape(5, pages)
    pool = torch.randint(0, 256, (5 * pages, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")
    want = pool.cpu().numpy().copy()
    kept = np.full((5, most), -1, np.int32)
    for b in range(5):
        kept[b, :count[b]] = np.sort(rng.permutation(far[b])[:count[b]])
        tr.keep(want, table[b], base[b], kept[b, :count[b]], Hkv, D, group, P)
    lens, err = ints([9999] * 5), error_word()
    q.mla_qcache_kv4_keep(cfg, ints(kept), ints(count), ints(base), ints(table), pool, lens, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and lens.tolist() == [a + n for a, n in zip(base, count)]
    assert np.array_equal(pool.cpu().numpy(), want)


def test_keep_reports_and_leaves_what_it_cannot_move():
    cfg = q.make_kv4_config(2, 64, page_size=16)
    start = torch.randint(0, 256, (6, q.kv4_page_bytes(cfg)), dtype=torch.uint8, device="cuda")

    def run(kept, count, base=(4, 4), table=((0, 1, 2), (3, 4, 5))):
        pool, lens, err = start.clone(), ints([40, 40]), error_word()
        q.mla_qcache_kv4_keep(cfg, ints(kept), ints(count), ints(base), ints(table), pool, lens, err)
        torch.cuda.synchronize()
        same = [torch.equal(pool[[x for x in t if 0 <= x < 6]], start[[x for x in t if 0 <= x < 6]]) for t in table]
        return int(err), lens.tolist(), same
    fine = [[0, 2, 5], [0, 3, -1]]
    assert run(fine, [3, 2]) == (0, [7, 6], [False, False])
    assert run([[0, 1, 2], [0, -1, -1]], [3, 1]) == (0, [7, 5], [True, True])  # nothing to move
    for first in ([0, 5, 2], [0, 2, 2], [-1, 2, 5], [0, 0, 1]):  # does not ascend
        assert run([first, fine[1]], [3, 2]) == (q.DEV_ROWS, [40, 6], [True, False]), first
    for count in (4, -1):
        assert run(fine, [count, 2]) == (q.DEV_ROWS, [40, 6], [True, False])
    assert run(fine, [3, 2], base=(-1, 4)) == (q.DEV_SEQ_OVERFLOW, [40, 6], [True, False])
    assert run(fine, [3, 2], base=(43, 4)) == (q.DEV_SEQ_OVERFLOW, [40, 6], [True, False])  # token 48 of 48
    assert run(fine, [0, 2], base=(49, 4)) == (q.DEV_SEQ_OVERFLOW, [40, 6], [True, False])
    assert run(fine, [0, 2], base=(48, 4)) == (0, [48, 6], [True, False])
    err, lens, same = run([[0, 2, 14], fine[1]], [3, 2], table=((0, 9, 2), (3, 4, 5)))  # token 18 lies in page 9
    assert (err, lens) == (q.DEV_BAD_PAGE, [7, 6]) and same == [False, False]

"""4-bit grouped-query cache on the GPU at the edges of its kernels: waits, page ids, windows, sizes of numbers and
row counts that the first tests leave out."""
import math

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests import kv4_paths
from tests.test_gpu_kv4 import Case, ints, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,n,lse", [(128, 64, False), (64, 64, True), (128, 130, True)])
def test_two_tiles_of_queries_over_many_segments_end_without_a_timeout(D, n, lse):
    """Over 128 rows, items cut over the SMs: a CTA goes through segments of one tile and of many. The warp that asks
    for later pages runs beside the others without holding them up; every call ends with its results and no error bit."""
    rng = np.random.default_rng(n)
    lens = rng.integers(n, 4500, 40)
    lens[:6] = [n, n + 1, 4499, 127 + n, 128 + n, 129 + n]
    c = Case([int(x) for x in lens], [n] * 40, Hkv=4 if n == 64 else 1, G=4, D=D, P=32, seed=n)
    ws = c.workspace()
    first = c.run(lse=lse, ws=ws)
    for _ in range(10):
        again = c.run(lse=lse, ws=ws)
        assert torch.equal(first[0], again[0]) and (not lse or torch.equal(first[1], again[1]))
    torch.cuda.synchronize()
    assert int(c.err) == 0 and not ws[:8192].any() and torch.isfinite(first[0]).all()


@pytest.mark.parametrize("n,G", [(1, 4), (6, 4), (20, 1), (20, 2), (40, 4)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30])
def test_windows_of_any_size_with_more_rows_than_tokens(n, G, window):
    """A window that no sequence fills is none; rows before the first token see nothing."""
    Case([0, max(1, n - 3), 300], [n, n, n], G=G, seed=n).check(window=window)


@pytest.mark.parametrize("n,G,D", [(1, 4, 128), (3, 8, 64), (6, 7, 128), (12, 10, 64), (40, 4, 128), (70, 2, 64)])
@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, "n_pages", 2 ** 31 - 1])
def test_any_id_outside_the_pool_is_a_bad_page(n, G, D, page):
    """Whatever the table holds in place of a page: its tokens are left out and the call says so, in each kernel."""
    c = Case([300, 70], [n, min(n, 2)], Hkv=2, G=G, D=D, P=32, seed=n)
    table, hide = c.table.copy(), [np.zeros(300, bool), np.zeros(70, bool)]
    for b, i in ((0, 1), (0, 6), (1, 0)):
        c.table[b, i] = c.n_pages if page == "n_pages" else page
        hide[b][32 * i:32 * i + 32] = True
    for lse in (True, False):
        c.err.zero_()
        out, l = c.run(lse=lse, scale=0.09)
        assert int(c.err) == q.DEV_BAD_PAGE
        bad, c.table = c.table, table
        kv4_paths.check(c, out, l, 0.09, hide=hide)
        c.table = bad


@pytest.mark.parametrize("n,G,D,lse", [(8, 4, 128, True), (9, 4, 128, True), (9, 4, 64, False), (10, 10, 128, False), (35, 4, 128, True),
                                       (35, 4, 64, False)])
@pytest.mark.parametrize("nats,at", [(16.3, 5), (17.4, 5), (17.4, 9000), (21.0, 300)])
def test_a_peak_above_many_small_weights(n, G, D, lse, nats, at):
    """One token `nats` above 16383 others of one score: what the others add up to is in the output, 1 in their values
    against 0 in the peak's. Their weights are far below the smallest normal FP16 number. Eighty sequences over the same
    pages: as many items as leave each whole, with one running max."""
    T, B = 16384, 80
    c = Case([1], [n], Hkv=1, G=G, D=D, P=256, seed=1)  # its table, pool and queries are replaced
    c.lens, c.table = [T], np.random.default_rng(2).permutation(T // 256).astype(np.int32)[None]
    c.n_pages = T // 256
    c.pool = torch.zeros((c.n_pages, q.kv4_page_bytes(c.cfg)), dtype=torch.uint8, device="cuda")
    k, v = torch.zeros((T, 1, D), dtype=c.t, device="cuda"), torch.ones((T, 1, D), dtype=c.t, device="cuda")
    k[at, 0, 0], v[at] = 15.0, 0.0
    q.mla_qcache_kv4_append(c.cfg, k, v, offsets([T]), ints([0]), T, ints(c.table), c.pool, c.err)
    c.lens, c.new, c.table = [T] * B, [n] * B, np.repeat(c.table, B, 0)
    c.q = torch.zeros((n * B, G, D), dtype=c.t, device="cuda")
    c.q[..., 0] = 1.0
    out, l = c.run(scale=nats / 15, lse=lse)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    if n * G > 32:  # (items of few rows are cut, each at other places)
        assert torch.equal(out, out[:n].repeat(B, 1, 1)) and (l is None or torch.equal(l, l[:n].repeat(B, 1)))
    c.lens, c.new = [T], [n]
    for at in (0, 37 * n, (B - 1) * n)[:1 if n * G > 32 else 3]:
        kv4_paths.check(c, out[at:at + n], None if l is None else l[at:at + n], nats / 15)


@pytest.mark.parametrize("n,G,D,group,lse", [(2, 4, 128, 64, True), (8, 4, 64, 32, True), (9, 4, 128, 128, False), (20, 5, 128, 32, True),
                                             (9, 4, 64, 64, True), (35, 4, 128, 64, True), (35, 4, 64, 32, True)])
@pytest.mark.parametrize("size", [1e-2, 1e-3, 3e-4, 1e-4, 1e-5, "large", "of every size"])
def test_keys_of_any_size_are_exact(n, G, D, group, lse, size):
    """Scales and minima down to the smallest FP16 numbers and up to the largest, one of them beside the other in a
    sequence, a token and a tile: where keys are promised exactly, scores of ten and more are right to float32."""
    rng = np.random.default_rng(n + D)
    c = Case([400, 130], [n, min(n, 3)], Hkv=2, G=G, D=D, group=group, P=32, seed=n)
    k = rng.standard_normal((530, 2, D))
    unit = 1.0
    if size == "large":  # a few groups whose scale is 4096 and more: 15 of it is beyond FP16
        k = k * 0.5
        k[::7, :, 3], k[::7, :, 5] = 64000.0, -63000.0
        k[5::11, 1, group - 1] = -50000.0
        k[5::11, 1, 0] = 40000.0
        unit = 2e4
    elif size == "of every size":
        k *= 10.0 ** rng.uniform(-5, 0, (530, 2, D // group, 1)).repeat(group, -1).reshape(530, 2, D)
        unit = 0.3
    else:
        k *= size
        unit = size
    kv = [torch.tensor(x, dtype=torch.float32).bfloat16().cuda() for x in (k, rng.standard_normal((530, 2, D)))]
    q.mla_qcache_kv4_append(c.cfg, *kv, offsets([400, 130]), ints([0, 0]), 400, ints(c.table), c.pool, c.err)
    scale = 1.2 / (unit * math.sqrt(D))  # queries of 2: scores of up to about ten
    out, l = c.run(scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    kv4_paths.check(c, out, l, scale)


@pytest.mark.parametrize("n,G,D,lse", [(2, 4, 128, True), (8, 4, 64, True), (9, 4, 128, True), (9, 4, 64, False), (35, 4, 128, True),
                                       (35, 4, 128, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_small_values_next_to_a_large_one_in_a_query(n, G, D, lse, dtype):
    """The first group of keys is zero and meets a query of 2^10; all that decides is in values of 2^-9 and less."""
    c = Case([300, 90], [n, min(n, 3)], Hkv=1, G=G, D=D, group=32, P=16, dtype=dtype, seed=n)
    rng = np.random.default_rng(n)
    k = rng.standard_normal((390, 1, D)) * 3
    k[..., :32] = 0
    kv = [torch.tensor(x, dtype=torch.float32).to(c.t).cuda() for x in (k, rng.standard_normal((390, 1, D)))]
    q.mla_qcache_kv4_append(c.cfg, *kv, offsets([300, 90]), ints([0, 0]), 300, ints(c.table), c.pool, c.err)
    c.q = (c.q.float() * 2.0 ** -10).to(c.t)
    c.q[..., 5] = 1024.0
    scale = 2.0 ** 9 / math.sqrt(D)
    out, l = c.run(scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    kv4_paths.check(c, out, l, scale)


@pytest.mark.parametrize("n,G,D,group,lse", [(3, 2, 128, 128, True), (5, 6, 64, 32, True), (9, 4, 128, 64, False), (40, 4, 128, 128, False),
                                             (40, 4, 64, 64, True)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 3e38, "nan among others", "both infinities"])
def test_values_that_are_no_numbers_stay_with_the_rows_that_see_them(n, G, D, group, lse, what):
    """The last of the new tokens has keys and values that are no numbers, or none of FP16's. The append says so; the rows
    in front of it, and those of the other sequence, get what they get without it."""
    lens, scale = [200, 77], 1 / math.sqrt(D)
    c = Case(lens, [n, min(n, 2)], Hkv=2, G=G, D=D, group=group, P=32, seed=n)
    rng = np.random.default_rng(n)
    good = torch.tensor(rng.standard_normal((2, 277, 2, D)), dtype=torch.float32).bfloat16().cuda()
    bad = good.clone()
    if what == "nan among others":
        bad[:, 199, :, 3::7] = float("nan")
    elif what == "both infinities":
        bad[:, 199, :, 0::2], bad[:, 199, :, 1::2] = float("inf"), -float("inf")
    else:
        bad[:, 199] = what
    results = []
    for kv in (good, bad):
        c.err.zero_()
        q.mla_qcache_kv4_append(c.cfg, kv[0], kv[1], offsets(lens), ints([0, 0]), 200, ints(c.table), c.pool, c.err)
        word = int(c.err)
        assert (word != 0) == (kv is bad) and word & ~(q.DEV_NONFINITE | q.DEV_RANGE) == 0
        c.err.zero_()
        out, l = c.run(lse=lse, scale=scale)
        assert int(c.err) == 0
        results.append((out, l))
    keep = torch.ones(sum(c.new), dtype=torch.bool)
    keep[n - 1] = False
    if what == 3e38:
        # held as 65504: a score that raises the running max of the rows beside it early, so that they round at other places;
        # every row is within its bound over what the cache holds
        kv4_paths.check(c, *results[1], scale)
        return
    assert torch.equal(results[0][0][keep], results[1][0][keep])
    assert not lse or torch.equal(results[0][1][keep], results[1][1][keep])


@pytest.mark.parametrize("n,G,D,lse", [(2, 4, 128, True), (8, 4, 64, True), (9, 4, 128, False), (9, 4, 64, True), (35, 4, 128, True),
                                       (35, 4, 128, False)])
@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** 116, 2.0 ** -90, 2.0 ** -104])
def test_queries_of_any_size(n, G, D, lse, size):
    """BF16 queries near both ends of their type, under a scale that makes scores of them."""
    c = Case([150, 40], [n, min(n, 3)], Hkv=2, G=G, D=D, P=16, seed=n)
    c.q = (c.q.float().clamp(-3.9, 3.9) * (size / 2)).to(c.t)
    scale = 2 / (size * math.sqrt(D))
    out, l = c.run(scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    kv4_paths.check(c, out, l, scale)


def test_a_flag_that_is_no_truth_value_is_refused():
    c = Case([40], [2], G=2)
    both = torch.tensor([True, False])
    with pytest.raises(RuntimeError, match="ambiguous"):
        c.run(causal=both)
    angle = torch.ones(50, 64, device="cuda")
    kv = torch.zeros(2, 1, 2, 128, dtype=c.t, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        q.mla_qcache_kv4_append(c.cfg, kv[0], kv[1], offsets([1]), ints([40]), 1, ints(c.table), c.pool, c.err, cos=angle, sin=angle,
                                interleaved=both)
    c.check()


@pytest.mark.parametrize("n,G,D,group,P", [
    (17, 1, 128, 128, 16), (8, 4, 64, 32, 64), (4, 8, 128, 64, 128), (32, 1, 128, 32, 128), (33, 1, 128, 128, 256), (12, 5, 64, 64, 16),
    (16, 4, 128, 32, 32), (13, 5, 128, 64, 64), (32, 4, 64, 32, 128), (32, 4, 128, 128, 64), (43, 3, 128, 32, 256), (37, 7, 64, 64, 256)])
@pytest.mark.parametrize("lse", [True, False])
def test_every_kernel_is_within_its_own_bound(n, G, D, group, P, lse):
    """Exact keys and values up to 32 rows, exact keys wherever they are promised: bounds without what does not apply."""
    for dtype in ("bf16", "fp16"):
        c = Case([n, 700, 1201, 3300], [n, n, 1, 2], Hkv=1, G=G, D=D, group=group, P=P, dtype=dtype, seed=n + D)
        for scale in (0.09, 0.5):
            out, l = c.run(lse=lse, scale=scale)
            torch.cuda.synchronize()
            assert int(c.err) == 0
            kv4_paths.check(c, out, l, scale)

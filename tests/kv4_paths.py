"""Bounds of the 4-bit attention by the kernel that a call takes, from the arithmetic that the header states:

few rows (max_q * heads of a kv head up to 32): exact keys, values and FP16 weights (kv4_ref.attention without tensor rows).
many: values rounded to FP16 (2^-11 of them, 2^-25 at the least), weights too (2^-11; they are scaled by 2^7, so that one below
  FP16's smallest normal number is off by at most 2^-25 2^-7 of the largest), keys exact; sums in float32.
many, keys rounded: also 2^-11 of every key in the scores. More than 128 rows (more than 32 at D = 64) without a log-sum-exp.

Queries enter as FP16 after a power of two: a value below 2^-20 of its row's largest is off by up to 2^-31 of that."""
import numpy as np
import torch

from tests import kv4_ref as ref


def path(rows_per_head, D, lse):
    if rows_per_head <= 32:
        return "few"
    return "many" if lse or (D == 128 and rows_per_head <= 128) else "many, keys rounded"


def query_error(q, k, scale, ok):
    """[n, Hq] how far the small values of a row of queries can move one of its scores."""
    n, Hq, D = q.shape
    top = np.abs(q).max(-1)  # [n, Hq]
    small = (np.abs(q) < 2.0 ** -20 * top[..., None]) & (q != 0)
    worst = np.zeros((n, Hq))
    for h in range(Hq):
        for i in range(n):
            if small[i, h].any() and ok[i].any():
                worst[i, h] = (np.abs(k[h // (Hq // k.shape[0])][ok[i]]) @ small[i, h]).max()
    return worst * top * 2.0 ** -31 * abs(scale)


def attention(q, k, v, vs, most, scale, ok, out_dtype, way):
    """As kv4_ref.attention, with the bound of `way`."""
    out, lse, bound = ref.attention(q, k, v, vs, most, scale, ok, out_dtype, False)
    if way == "few":
        return out, lse, bound + query_error(q, k, scale, ok)[..., None] * 2 * np.abs(v).max(initial=0)
    n, Hq, D = q.shape
    G, T, half = Hq // k.shape[0], k.shape[1], torch.finfo(out_dtype).eps / 2
    off = query_error(q, k, scale, ok)
    for h in range(Hq):
        kk, vv = k[h // G], np.abs(v[h // G])
        s = (q[:, h] @ kk.T) * scale
        mag = (np.abs(q[:, h]) @ np.abs(kk).T) * abs(scale)
        for i in range(n):
            m = ok[i]
            if not m.any():
                continue
            p = np.exp(s[i, m] - lse[i, h])
            e = 2 * D * 2.0 ** -24 * mag[i, m] + 2.0 ** -20 + T * 2.0 ** -24 + off[i, h]
            if way != "many":
                e = e + 2.0 ** -11 * mag[i, m]
            pv = p @ vv[m]
            b = (p * e) @ vv[m] + (p @ e) * pv + (2.0 ** -10 + 2 * T * 2.0 ** -24) * pv
            b += 2.0 ** -25 + T * 2.0 ** -32 * vv[m].max()
            bound[i, h] = b * (1 + half) + half * np.abs(out[i, h]) + 2.0 ** -24
    return out, lse, bound


def check(c, out, lse, scale, window=0, causal=True, hide=None, max_q=None):
    """Compares a call's results with the statement in 64 bits; c: the test's Case, hide: [sequences][tokens] left out."""
    pool, r = c.pool.cpu().numpy(), 0
    way = path((max_q or max(c.new)) * (c.Hq // c.Hkv), c.D, lse is not None)
    for b, (T, n) in enumerate(zip(c.lens, c.new)):
        k, v, vs, most = ref.read_sequence(pool, c.table[b], T, c.Hkv, c.D, c.group, c.P)
        ok = ref.seen(T, n, causal, window)
        if hide is not None:
            ok &= ~hide[b][None, :T]
        qq = c.q[r:r + n].double().cpu().numpy()
        want, wl, bound = attention(qq, k, v, vs, most, scale, ok, c.t, way)
        got = out[r:r + n].double().cpu().numpy()
        assert np.isfinite(got).all()
        off = np.abs(got - want)
        assert (off <= bound).all(), f"{way}, sequence {b}: {(off - bound).max():.3e} beyond the bound ({(off / bound).max():.2f} of it)"
        if lse is not None:
            gl = lse[r:r + n].double().cpu().numpy()
            fin = np.isfinite(wl)
            assert np.array_equal(np.isneginf(gl), ~fin)
            far = np.abs(gl[fin] - wl[fin])
            assert (far <= (ref.lse_bound(qq, k, scale, ok) + query_error(qq, k, scale, ok))[fin]).all(), f"{way}, sequence {b}: log-sum-exp off by {far.max():.3e}"
        r += n

"""Plain statement in 64 bits of the grouped-query cache in 4 bits, from the formulas of the header:
page layout, quantizer, rotation, attention with its error bound. CPU only, loops where they are clear."""
import math

import numpy as np
import torch

F64 = torch.float64


def head_bytes(D, group, P):
    return P * (D + 8 * (D // group))


def key_nibble(c, D):
    return 8 * ((c % 32 // 8) * (D // 32) + c // 32) + c % 8


def value_nibble(c, D):
    return 8 * ((c % 8) * (D // 64) + c // 64) + 4 * (c // 8 % 2) + c // 16 % 4


def half_down(x):
    """Largest FP16 value <= x (numpy float64 array; zero is +0)."""
    with np.errstate(over="ignore"):
        h = x.astype(np.float16)
    h = np.where(h.astype(np.float64) > x, np.nextafter(h, np.float16(-np.inf)), h)
    return np.where(h == 0, np.float16(0), h)


def half_up(x):
    return -half_down(-x) + np.float16(0)


def quantize(x, group):
    """x [..., D] float64 -> codes, scale, minimum (numpy)."""
    v = x.reshape(*x.shape[:-1], -1, group)
    lo, hi = v.min(-1), v.max(-1)
    m = half_down(lo)
    s = half_up((hi - m.astype(np.float64)) / 15)
    m64, s64 = m.astype(np.float64)[..., None], s.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.rint((v - m64) / s64)  # ties to the even code; differences and midpoints are exact in 64 bits
    n = np.where(s64 > 0, np.clip(n, 0, 15), 0).astype(np.uint8)
    return n.reshape(x.shape), s, m


def values(codes, s, m, group):
    v = codes.reshape(*codes.shape[:-1], -1, group).astype(np.float64)
    return (v * s.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]).reshape(codes.shape)


def rotate32(x, cos, sin, interleaved):
    """Rotation in float32, every product and sum rounded: x [rows, heads, D] float32 numpy, cos/sin [rows, half]."""
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    y = x.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def pack_rows(codes, nibble, D):
    out = np.zeros(codes.shape[:-1] + (D // 2,), np.uint8)
    for c in range(D):
        i = nibble(c, D)
        out[..., i // 2] |= codes[..., c] << (4 * (i % 2))
    return out


def unpack_rows(rows, nibble, D):
    return np.stack([rows[..., nibble(c, D) // 2] >> (4 * (nibble(c, D) % 2)) & 15 for c in range(D)], -1)


def put_token(pool, page, t, h, D, group, P, key, val):
    """Stores one token of one head: key, val = (codes [D], scale [G], min [G])."""
    r = pool[page, h * head_bytes(D, group, P):(h + 1) * head_bytes(D, group, P)]
    r[t * D // 2:(t + 1) * D // 2] = pack_rows(key[0], key_nibble, D)
    r[P * D // 2 + t * D // 2:P * D // 2 + (t + 1) * D // 2] = pack_rows(val[0], value_nibble, D)
    num = np.stack([key[1], key[2], val[1], val[2]], -1).astype(np.float16)
    G = D // group
    r[P * D + t * G * 8:P * D + (t + 1) * G * 8] = np.frombuffer(num.tobytes(), np.uint8)


def read_sequence(pool, table_row, T, Hkv, D, group, P):
    """Keys and values [Hkv, T, D] (float64), the part of each value that its code carries, and each head's largest
    value scale."""
    pages = table_row[:-(-T // P)] if T else table_row[:0]
    k, v, vs = (np.zeros((Hkv, T, D)) for _ in range(3))
    most = np.zeros(Hkv)
    for h in range(Hkv):
        r = pool[pages, h * head_bytes(D, group, P):(h + 1) * head_bytes(D, group, P)]
        cut = lambda a, b, w: r[:, a:b].reshape(-1, w)[:T]  # noqa: E731
        num = np.ascontiguousarray(cut(P * D, P * D + P * 8 * (D // group), 8 * (D // group))).view(np.float16)
        num = num.reshape(T, D // group, 4).astype(np.float64).repeat(group, 1)
        kc = unpack_rows(cut(0, P * D // 2, D // 2), key_nibble, D)
        vc = unpack_rows(cut(P * D // 2, P * D, D // 2), value_nibble, D)
        k[h] = kc * num[..., 0] + num[..., 1]
        vs[h] = vc * num[..., 2]
        v[h] = vs[h] + num[..., 3]
        most[h] = num[..., 2].max(initial=0)
    return k, v, vs, most


def seen(T, n, causal, window):
    """[n, T] which tokens each of the last n rows sees."""
    pos = np.arange(T - n, T)[:, None]
    t = np.arange(T)[None]
    ok = np.ones((n, T), bool)
    if causal:
        ok = t <= pos
        if window:
            ok &= t > pos - window
    return ok


def attention(q, k, v, vs, most, scale, ok, out_dtype, tensor_rows):
    """q [n, Hq, D] float64; k, v, vs [Hkv, T, D]. Returns out, lse [n, Hq(, D)] in 64 bits and the bound of the
    output's error:

    few rows (tensor_rows False): scores are exact products summed in float32, so a weight's relative error is at
      most e = 2 D 2^-24 |q|.|k| scale + 2^-20 (the exponential, scaling); the weight times its scale is rounded to
      FP16, 2^-11 of sum p vs n; every sum of T terms in float32 adds less than T 2^-24 of its terms. FP16 ends at
      2^-14: below, a weight is off by up to half of its last step, 2^-25, in a unit (the power of two that scales
      the weights) of at most a sixteenth of the largest value scale, times a code of at most 15, over a denominator
      of at least 1 (the reference of the exponentials is a score that was seen): T 15 2^-29 of that scale.
    many rows: also keys and values rounded to FP16 (2^-11 of them, keys through the score) and weights (2^-11).
    Numerator and denominator both carry e; the result is rounded once to the output's type."""
    n, Hq, D = q.shape
    Hkv, T, _ = k.shape
    G = Hq // Hkv
    out, lse, bound = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    half = torch.finfo(out_dtype).eps / 2
    for h in range(Hq):
        kk, vv, ss = k[h // G], v[h // G], vs[h // G]
        s = (q[:, h] @ kk.T) * scale
        mag = (np.abs(q[:, h]) @ np.abs(kk).T) * abs(scale)
        for i in range(n):
            m = ok[i]
            if not m.any():
                continue
            top = s[i, m].max()
            p = np.exp(s[i, m] - top)
            L = p.sum()
            lse[i, h] = top + math.log(L)
            p /= L
            out[i, h] = p @ vv[m]
            e = 2 * D * 2.0 ** -24 * mag[i, m] + 2.0 ** -20 + T * 2.0 ** -24
            b = (p * e) @ np.abs(vv[m]) + (p @ e) * (p @ np.abs(vv[m]))
            b += (T * 2.0 ** -24) * (p @ ss[m] + p @ np.abs(vv[m] - ss[m]))
            if tensor_rows:
                ek = 2.0 ** -11 * mag[i, m]  # a key off by 2^-11 of itself
                b += (p * ek) @ np.abs(vv[m]) + (p @ ek) * (p @ np.abs(vv[m])) + 2.0 ** -10 * (p @ np.abs(vv[m]))
            else:
                b += 2.0 ** -11 * (p @ np.abs(ss[m])) + T * 15 * 2.0 ** -29 * most[h // G]
            bound[i, h] = b * (1 + half) + half * np.abs(out[i, h]) + 2.0 ** -24
    return out, lse, bound


def lse_bound(q, k, scale, ok, rows_exact=True):
    """|lse error| of scores summed in float32 (keys exact, or in two FP16 parts): the largest score error, plus the
    logarithm and sum in float32."""
    n, Hq, D = q.shape
    G = Hq // k.shape[0]
    b = np.zeros((n, Hq))
    for h in range(Hq):
        mag = (np.abs(q[:, h]) @ np.abs(k[h // G]).T) * abs(scale)
        for i in range(n):
            if ok[i].any():
                b[i, h] = (2 * D * 2.0 ** -24 + 2.0 ** -21) * mag[i, ok[i]].max() + 2.0 ** -19 + k.shape[1] * 2.0 ** -24
    return b

"""Plain statements of what trees of drafted tokens need: masks, what a node sees, verification in exact rational numbers, and
moving the kept nodes. CPU only, loops where they are clear."""
from fractions import Fraction

import numpy as np
import torch


def masks(parents):
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def random_parents(rng, n, reach=6):
    return ([-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, n)])[:n]


def mask_tensor(ms, words, device="cuda"):
    signed = lambda x: x - (1 << 64) if x >> 63 else x  # noqa: E731
    return torch.tensor([[signed(m >> 64 * w & (1 << 64) - 1) for w in range(words)] for m in ms], dtype=torch.int64,
                        device=device).reshape(len(ms), words)


def seen(T, base, ms, words, window):
    """[rows, T] which tokens rows with these masks see."""
    ok = np.zeros((len(ms), T), bool)
    for i, m in enumerate(ms):
        m &= (1 << 64 * words) - 1
        pos = base + bin(m).count("1") - 1
        for t in range(T):
            ok[i, t] = (not window or t > pos - window) if t < base else t - base < 64 * words and m >> (t - base) & 1
    return ok


def parents_of(ms):
    out = []
    for i, m in enumerate(ms):
        below = m & ((1 << i) - 1)
        out.append(below.bit_length() - 1)
    return out


def _mass(x):
    x = float(x)
    return Fraction(x) if np.isfinite(x) and x > 0 else Fraction(0)


def verify_sampled(target, draft, tokens, parents, u_accept, u_sample):
    """One sequence: (kept, new tokens), in rational numbers. target, draft: [rows][vocab] float32 (draft may be None)."""
    V = target.shape[1]
    at, kept, new = 0, [0], []

    def left(c, gone):
        p = [_mass(x) for x in target[at]]
        if draft is None:
            return [Fraction(0) if j in gone else x for j, x in enumerate(p)]
        return [max(x - c * _mass(y), Fraction(0)) for x, y in zip(p, draft[at])]
    while True:
        c, Z, gone, taken = Fraction(0), Fraction(1), set(), -1
        for x in range(at + 1, len(parents)):
            t = int(tokens[x])
            if parents[x] != at or not 0 <= t < V:
                continue
            u, p = Fraction(float(u_accept[x])), _mass(target[at][t])
            if draft is None:
                ok = u * Z < (0 if t in gone else p)
            else:
                q = _mass(draft[at][t])
                ok = u * q * Z < max(p - c * q, 0)
            if ok:
                taken = x
                break
            if draft is None:
                if t not in gone:
                    Z -= p
                gone.add(t)
            else:
                c += Z
                Z = sum(left(c, gone))
        if taken < 0:
            break
        at = taken
        kept.append(at)
        new.append(int(tokens[at]))
    rest = left(c, gone)
    if not any(rest):
        rest = [_mass(x) for x in target[at]]
    total = sum(rest)
    if not total:
        return kept, new + [-1]
    goal, run, token = Fraction(float(u_sample)) * total, Fraction(0), -1
    for j, x in enumerate(rest):
        if x > 0:
            token = j
            run += x
            if run > goal:
                break
    return kept, new + [token]


def verify_greedy(logits, tokens, parents):
    """One sequence: logits [rows][vocab] float64."""
    at, kept, new = 0, [0], []
    while True:
        row = logits[at]
        fine = ~np.isnan(row)
        best = int(np.argmax(np.where(fine, row, -np.inf))) if fine.any() else -1  # the first of equal ones
        if fine.any() and np.isneginf(row[fine].max()):
            best = int(np.argmax(fine))
        new.append(best)
        nxt = [x for x in range(at + 1, len(parents)) if parents[x] == at and best >= 0 and int(tokens[x]) == best]
        if not nxt:
            return kept, new
        at = nxt[0]
        kept.append(at)


def token_bytes(pool, page, t, h, D, group, P):
    """Views of the bytes of one token of one head: key codes, value codes, numbers."""
    G = D // group
    r = pool[page, h * P * (D + 8 * G):(h + 1) * P * (D + 8 * G)]
    return (r[t * D // 2:(t + 1) * D // 2], r[P * D // 2 + t * D // 2:P * D // 2 + (t + 1) * D // 2],
            r[P * D + t * 8 * G:P * D + (t + 1) * 8 * G])


def keep(pool, table, base, kept, Hkv, D, group, P):
    """Moves one sequence's tokens base + kept[i] to base + i (numpy, in place)."""
    for h in range(Hkv):
        held = [[x.copy() for x in token_bytes(pool, table[(base + k) // P], (base + k) % P, h, D, group, P)] for k in kept]
        for i, parts in enumerate(held):
            for to, x in zip(token_bytes(pool, table[(base + i) // P], (base + i) % P, h, D, group, P), parts):
                to[:] = x

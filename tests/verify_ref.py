"""Sampled verification in whole numbers of any length, for rows as long as real vocabularies: what tree_ref.verify_sampled states in
fractions, a row at a time. CPU only."""
import bisect
from fractions import Fraction

import numpy as np

UNIT = 149  # every float32 is a whole number of 2^-149


def whole(row):
    """Entries of a float32 row that count (positive and finite) as whole numbers of 2^-149, the others 0."""
    x = np.where(np.isfinite(row) & (row > 0), row, 0).astype(np.float64)
    m, e = np.frexp(x)
    out = np.empty(len(x), object)
    out[:] = [int(a) << int(b) if a else 0 for a, b in zip((m * 2.0 ** 24).astype(np.int64), e + (UNIT - 24))]
    return out


class Rows:
    """whole() of the rows that are asked for, each once."""

    def __init__(self, rows):
        self.rows, self.held = rows, {}

    def __getitem__(self, r):
        if r not in self.held:
            self.held[r] = whole(self.rows[r])
        return self.held[r]


def walk(target, draft, tokens, parents, u_accept, first=0):
    """One sequence, its rows first, first + 1, .. of target and draft (Rows, draft may be None): kept, accepted tokens, and what is left
    of the last node's row in a unit of its own."""
    V = target.rows.shape[1]
    at, kept, new = 0, [0], []
    while True:
        p, d = target[first + at], None if draft is None else draft[first + at]
        c, steps, Z, gone, taken = 0, 0, Fraction(1), set(), -1  # c in units of 2^(-149 steps)

        def left():
            if d is None:
                out = p.copy()
                out[list(gone)] = 0
                return out
            return np.maximum(p * (1 << UNIT * steps) - d * c, 0) if c else p
        for x in range(at + 1, len(parents)):
            t = int(tokens[x])
            if parents[x] != at or not 0 <= t < V:
                continue
            u = Fraction(float(u_accept[x]))
            if d is None:
                ok = u * Z < (0 if t in gone else Fraction(p[t], 1 << UNIT))
            else:
                ok = u * Fraction(d[t], 1 << UNIT) * Z < max(Fraction(p[t], 1 << UNIT) - Fraction(c, 1 << UNIT * steps) * Fraction(d[t], 1 << UNIT), 0)
            if ok:
                taken = x
                break
            if d is None:
                if t not in gone:
                    Z -= Fraction(p[t], 1 << UNIT)
                gone.add(t)
            elif steps == 0 and c == 0:  # c = 1 to begin with, whose row has the unit of p and d
                c, Z = 1, None
                Z = Fraction(sum(left()), 1 << UNIT)
            else:
                steps += 1
                c = (c << UNIT) + int(Z * (1 << UNIT * steps))  # Z is a whole number of that unit
                Z = Fraction(sum(left()), 1 << UNIT * (steps + 1))
        if taken < 0:
            rest = left()
            return kept, new, rest if rest.any() else p
        at = taken
        kept.append(at)
        new.append(int(tokens[at]))


class Sampler:
    """The new token of a row that is left, for one random number after the other."""

    def __init__(self, rest):
        self.rest, self.upto = rest, list(np.cumsum(rest))

    def __call__(self, u):
        total = self.upto[-1]
        if not total:
            return -1
        a = Fraction(float(u)) * total
        j = bisect.bisect_right(self.upto, a.numerator // a.denominator)  # whole numbers: above a is above its floor
        return j if j < len(self.upto) else int(np.flatnonzero(self.rest)[-1])

    def number_for(self, j):
        """A random number in whose share entry j lies, or the nearest behind it with something in it (float32: nearly)."""
        some = np.flatnonzero(self.rest)
        j = int(some[min(np.searchsorted(some, j), len(some) - 1)])
        u = np.float32(float(Fraction(2 * self.upto[j] - self.rest[j], 2 * self.upto[-1])))
        return min(u, np.float32(1 - 2.0 ** -24))

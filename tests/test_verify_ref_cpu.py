"""The statement of sampled verification in whole numbers is the one in fractions."""
import numpy as np
import pytest

from tests import tree_ref as tr, verify_ref as vr


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1, 3, 20])
def test_both_statements_are_one(V, drawn):
    rng = np.random.default_rng(V)
    seen = set()
    for case in range(60):
        n = int(rng.integers(1, 9))
        parents = tr.random_parents(rng, n, 4)
        z = rng.standard_normal((n, V))
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        p, d = soft(z), soft(z + 1.5 * rng.standard_normal((n, V)))
        if case % 7 == 0:
            p[:, 0], d[:, -1] = np.nan, 0
        tokens, ua = rng.integers(-1, V + 1, n), np.where(rng.random(n) < 0.5, 0.999, rng.random(n)).astype(np.float32)
        draft = d if drawn else None
        kept, new, rest = vr.walk(vr.Rows(p), None if draft is None else vr.Rows(d), tokens, parents, ua)
        sampler = vr.Sampler(rest)
        for u in (0.0, rng.random(), 1 - 2.0 ** -24, sampler.number_for(V // 2) if rest.any() else 0.5):
            u = np.float32(u)
            want = tr.verify_sampled(p, draft, tokens, parents, ua, u)
            assert (kept, new + [sampler(u)]) == want
        seen.add(len(kept))
    assert V == 1 or len(seen) > 1

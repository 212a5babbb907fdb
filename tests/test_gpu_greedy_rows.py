"""Greedy verification in both of its ways, up to eight rows of a sequence at once and one row after the other, against the plain statement
and against each other."""
import numpy as np
import pytest
import torch

from tests import tree_ref as tr
from tests.test_gpu_verify import call_greedy, check_greedy

pytestmark = pytest.mark.gpu
F32 = torch.float32


def greedy_inputs(rng, sizes, V, dtype, chain):
    ps = [[i - 1 for i in range(n)] if chain else tr.random_parents(rng, n, 3) for n in sizes]
    x = torch.tensor(np.round(rng.standard_normal((sum(sizes), V)) * 2) / 2, dtype=F32).to(dtype).cuda()  # many equal ones
    best = x.double().cpu().numpy().argmax(1)
    t, r = np.zeros(sum(sizes), np.int64), 0
    for p in ps:
        for i, a in enumerate(p):
            t[r + i] = best[r + a] if a >= 0 and rng.random() < 0.8 else int(rng.integers(-1, V + 1))
        r += len(p)
    return ps, x, t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V,times", [(1, 1), (2, 5), (9, 1), (31, 5), (255, 1), (1000, 5), (4099, 1), (4099, 5), (40001, 1), (40001, 5), (150001, 1)])
@pytest.mark.parametrize("chain", [True, False])
def test_greedy_of_up_to_eight_rows(dtype, V, times, chain):
    """Every count of rows that are taken at once, with idle parts and without; a bound of nine takes them one after the other."""
    rng = np.random.default_rng(V + times)
    sizes = [1, 2, 0, 3, 4, 5, 7, 8, 6] * times
    ps, x, t = greedy_inputs(rng, sizes, V, dtype, chain)
    ms = None if chain else [m for p in ps for m in (tr.masks(p) if p else [])]
    got = call_greedy(x, t, sizes, ms, max_rows=8)
    assert got[3] == 0
    check_greedy(x, t, ps, got)
    after = call_greedy(x, t, sizes, ms, max_rows=9)
    assert after[3] == 0 and after[2] == got[2]
    assert np.array_equal(after[0][:, :8], got[0]) and np.array_equal(after[1][:, :8], got[1])
    wide = torch.full((len(x), V + 5), float("inf"), dtype=dtype, device="cuda")
    wide[:, 3:3 + V] = x
    odd = call_greedy(wide[:, 3:3 + V], t, sizes, ms, max_rows=8)
    assert odd[2] == got[2] and np.array_equal(odd[0], got[0]) and np.array_equal(odd[1], got[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [50, 40001, 150001])
@pytest.mark.parametrize("max_rows", [4, 9])
def test_greedy_where_little_is_allowed(dtype, V, max_rows):
    """Rows of -inf but for a few entries, or for none, and NaN in between: decoding under constraints."""
    rng = np.random.default_rng(V + max_rows)
    B, n = 5, 4
    x = torch.full((B * n, V), -float("inf"), dtype=dtype, device="cuda")
    t = np.zeros(B * n, np.int64)
    for r in range(B * n):
        at = sorted(int(a) for a in rng.integers(0, V, 3))
        if r % 5 < 4:
            x[r, at] = torch.tensor([1.0, 1.0, -2.0], dtype=dtype, device="cuda") if r % 5 else torch.tensor([-float("inf")] * 3, dtype=dtype, device="cuda")
        else:  # NaN before the first number
            x[r, :at[1]] = float("nan")
        if r % n < n - 1:
            row = x[r].double().cpu().numpy()
            fine = ~np.isnan(row)
            t[r + 1] = int(np.argmax(np.where(fine, row, -np.inf))) if np.isfinite(row[fine]).any() else int(np.argmax(fine))
    chain = [list(range(-1, n - 1))] * B
    got = call_greedy(x, t, [n] * B, max_rows=max_rows)
    assert got[3] == 0
    check_greedy(x, t, chain, got)

"""Verification where the number of threads changes (as many sequences as the GPU holds clusters, and one more), and a first call that is
captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import tree_ref as tr
from tests.test_gpu_verify import call_greedy, call_sampled, check_greedy, check_sampled, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drawn", [True, False])
def test_results_do_not_go_by_the_number_of_sequences(drawn):
    """The same sequences, alone and among ever more of them."""
    rng = np.random.default_rng(3)
    n, V = 4, 700
    ps, p, d, t, ua, us = make(rng, [n] * 5, V, True, drawn, near=1.0)
    seen = []
    for B in (5, 20, 35, 40, 75, 150):
        times = B // 5
        wide = lambda x: None if x is None else torch.tensor(np.tile(x, (times, 1))).cuda()  # noqa: E731
        got = call_sampled(wide(p), wide(d), np.tile(t, times), [n] * B, np.tile(ua, times), np.tile(us, times))
        assert got[3] == 0
        check_sampled(p, d, t, ps, ua, us, (got[0][:5], got[1][:5], got[2][:5], 0), n)
        for k in range(times):
            assert np.array_equal(got[1][5 * k:5 * k + 5], got[1][:5]) and np.array_equal(got[0][5 * k:5 * k + 5], got[0][:5])
        seen.append(got[1][:5].tolist())
    assert all(s == seen[0] for s in seen)


@pytest.mark.parametrize("B", [36, 37, 38, 74, 75])
def test_greedy_of_as_many_sequences_as_fit(B):
    rng = np.random.default_rng(B)
    n, V = 3, 501
    x = torch.tensor(np.round(rng.standard_normal((B * n, V))), dtype=torch.float32).half().cuda()
    best = x.double().cpu().numpy().argmax(1)
    t = np.array([best[r - 1] if r % n and rng.random() < 0.7 else 0 for r in range(B * n)])
    chain = [list(range(-1, n - 1))] * B
    check_greedy(x, t, chain, call_greedy(x, t, [n] * B))
    check_greedy(x, t, chain, call_greedy(x, t, [n] * B, [m for p in chain for m in tr.masks(p)], max_rows=9))


def test_a_first_call_may_be_captured():
    """A process whose first verification is captured: what the launches ask the device for is allowed there."""
    code = """
import torch
import bit_mla_kv_qcache_gb300 as q
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
p = torch.zeros(2, 100, device="cuda")
p[:, 42] = 1
tok, cu, u = i(0, 42), i(0, 2), torch.full((2,), 0.5, device="cuda")
kept, new, n, err = i(0, 0).view(1, 2), i(0, 0).view(1, 2), i(0), i(0)
half = p.half()
q.lib()
torch.cuda.synchronize()
for call in (lambda: q.mla_qcache_verify_sampled(p, tok, cu, 2, u, u[:1], kept, new, n, err),
             lambda: q.mla_qcache_verify_greedy(half, tok, cu, 2, kept, new, n, err)):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    new.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert new.tolist() == [[42, 42]] and n.tolist() == [2] and int(err) == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]

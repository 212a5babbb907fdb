"""The launch that joins the parts of cut items, on parts laid out here: an item of which a part was not stored, as after a wait that ran
out, stays as it is; what an earlier call left in the workspace is not taken for it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from bit_mla_kv_qcache_gb300 import build

pytestmark = pytest.mark.gpu
ROOM = 7.0  # weights and their sums carry 2^7


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    q.lib()
    here, lib = os.path.dirname(os.path.abspath(__file__)), str(tmp_path_factory.mktemp("join") / "join.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    cmd = ["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", build.CSRC, "-I", os.path.join(cuda, "include"),
           os.path.join(here, "join_harness.cpp"), "-o", lib, "-L", build.PKG, "-l:" + os.path.basename(build.LIB), "-Wl,-rpath," + build.PKG]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(lib).join_parts
    i, p = ctypes.c_int, ctypes.c_void_p
    f.argtypes, f.restype = [i, i, i, i, p, p, p, i, p, p, p], i
    return f


@pytest.mark.parametrize("D,rows,G,parts", [(128, 64, 4, 3), (64, 128, 8, 5), (128, 256, 8, 32), (64, 64, 16, 20), (64, 256, 2, 2)])
def test_items_with_a_part_that_is_missing_stay(join, D, rows, G, parts):
    rng = np.random.default_rng(D + rows)
    ctas, first = parts + 3, 2  # the item begins at CTA 2; CTA 2 ends an earlier one of which nobody asks
    n = rows // G  # rows of queries
    live = n * G - 3
    part_o = torch.tensor(rng.standard_normal((2 * ctas, rows, D)), dtype=torch.float32, device="cuda")
    ml = np.stack([rng.standard_normal((2 * ctas, rows)), 2.0 ** ROOM * rng.uniform(1, 5, (2 * ctas, rows))], -1)
    part_ml = torch.tensor(ml, dtype=torch.float32, device="cuda")
    slots = [2 * first + 1] + [2 * (first + i) for i in range(1, parts)]

    def run(missing):
        joined = np.zeros((ctas, 5), np.int32)
        joined[first] = [0, 0, parts, 0, live]
        marked = part_ml.clone()
        marked[2 * first] = marked[slots[-1] + 1] = torch.tensor([-1e30, -1.0])  # of other items
        for i in missing:
            marked[slots[i]] = torch.tensor([-1e30, -1.0])
        out = torch.full((n, G, D), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((n, G), 7.0, device="cuda")
        j = torch.tensor(joined, device="cuda")
        assert join(ctas, rows, D, G, part_o.data_ptr(), marked.data_ptr(), j.data_ptr(), 1, out.data_ptr(), lse.data_ptr(),
                    torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return out.view(n * G, D), lse.view(n * G)
    out, lse = run([])
    m, l = part_ml.double().cpu().numpy()[slots, :, 0], part_ml.double().cpu().numpy()[slots, :, 1]
    M = m.max(0)
    L = (np.exp2(m - M) * l).sum(0)
    want = (np.exp2(m - M) * l / L)[..., None]  # each part's share; the sums in it are not divided by its own
    want = (want / l[..., None] * part_o.double().cpu().numpy()[slots]).sum(0)
    assert np.abs(lse[:live].double().cpu().numpy() - (M + np.log2(L) - ROOM)[:live] * np.log(2)).max() < 1e-5
    # columns come in the order in which codes were unpacked: the same values
    assert np.abs(np.sort(out[:live].double().cpu().numpy(), 1) - np.sort(want[:live], 1)).max() <= 2.0 ** -11 * np.abs(want).max() + 1e-5
    assert (out[live:] == 7).all() and (lse[live:] == 7).all()
    for missing in ([0], [1], [parts - 1], list(range(parts))):
        out, lse = run(missing)
        assert (out == 7).all() and (lse == 7).all(), missing

"""Calls of the trees' entry points that are refused before any launch: results over the error word."""
import ctypes

import bit_mla_kv_qcache_gb300 as q
from tests.test_kv4_cpu import P16, PFAR, lib  # noqa: F401
from tests.test_tree_cpu import PB, PC, _greedy, _sampled


def test_results_over_the_error_word_are_refused(lib):  # noqa: F811
    at = lambda p, n: ctypes.c_void_p(p.value + n)  # noqa: E731
    for call in (_sampled, _greedy):  # lists of 2 x 3 numbers, counts of 2
        for err in (PC, at(PC, 20), at(PC, 4096), at(PC, 4096 + 20), at(PC, 8192), at(PC, 8196)):
            assert call(lib, err=err) == -3, err
    cfg = q.make_kv4_config(2, page_size=16)
    for err in (PB, at(PB, 4), PFAR, at(PFAR, 8 * q.kv4_page_bytes(cfg) - 4)):
        assert lib.mla_qcache_kv4_keep(ctypes.byref(cfg), 2, P16, 8, P16, P16, P16, 4, PFAR, 8, PB, err, None) == -3
    for err in (PFAR, at(PFAR, 28)):
        assert lib.mla_qcache_tree_mask(2, 4, P16, P16, 8, 1, PFAR, err, None) == -3

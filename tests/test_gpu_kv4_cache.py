"""KV4Cache beside other streams and in captured graphs: its workspaces, its results and its lengths."""
import numpy as np
import pytest
import torch

import bit_mla_kv_qcache_gb300 as q
from tests.test_gpu_kv4 import offsets

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def rows(rng, n, heads):
    return torch.tensor(rng.standard_normal((n, heads, 128)), dtype=torch.float32).bfloat16().cuda()


def filled(lens, Hkv=2, seed=0, P=64, spare=2):
    """A cache that holds `lens` tokens; long sequences are cut into parts, so that calls use the counters."""
    rng = np.random.default_rng(seed)
    cache = q.KV4Cache(q.make_kv4_config(Hkv, page_size=P), len(lens), -(-max(lens) // P) + spare)
    cache.append(rows(rng, sum(lens), Hkv), rows(rng, sum(lens), Hkv), offsets(lens), max(lens))
    torch.cuda.synchronize()
    return cache, rng


def test_first_call_on_a_stream_of_its_own_while_another_is_busy():
    """The workspace is zeroed, and the output allocated, on the stream that uses them: nothing else orders them."""
    for max_q, n in ((1, 1), (30, 30)):
        cache, rng = filled([5000, 700], seed=max_q)
        query, cu = rows(rng, 2 * n, 8), offsets([n, n])
        want = cache.attend(query, SCALE, cu_q=cu, max_q=max_q)
        torch.cuda.synchronize()
        other, _ = filled([5000, 700], seed=max_q)
        other.pool, other.seq_lens = cache.pool, cache.seq_lens
        s = torch.cuda.Stream()
        dirt = torch.full((other.workspace(8, max_q).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
        other._ws.clear()
        del dirt
        torch.cuda.synchronize()
        torch.cuda._sleep(1 << 28)  # the current stream is busy for a while
        got = other.attend(query, SCALE, cu_q=cu, max_q=max_q, stream=s)
        s.synchronize()
        assert torch.cuda.current_stream().query() is False  # it did not wait for the other stream
        torch.cuda.synchronize()
        assert torch.equal(got, want) and cache.error_bits() == 0 == other.error_bits()


def test_two_streams_at_once_have_workspaces_of_their_own():
    cache, rng = filled([6000, 900], seed=3)
    a, b = rows(rng, 2, 8), rows(rng, 2, 8)
    want = [cache.attend(x, SCALE).clone() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    places = {cache.workspace(8, 1, s).data_ptr() for s in streams} | {cache.workspace(8, 1).data_ptr()}
    assert len(places) == 3
    assert cache.workspace(8, 1, streams[0]).data_ptr() in places  # kept
    for _ in range(50):
        got = [cache.attend(x, SCALE, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and cache.error_bits() == 0


def test_captured_call_outlives_larger_calls():
    """A captured step is replayed after larger calls through the same object have replaced its workspaces: it writes
    nothing into memory that others have since been given."""
    cache, rng = filled([5000, 700], seed=4)
    query, prompt, cu = rows(rng, 2, 8), rows(rng, 140, 8), offsets([70, 70])
    want = cache.attend(query, SCALE).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cache.attend(query, SCALE)
    cache.attend(prompt, SCALE, cu_q=cu, max_q=70)
    torch.cuda.synchronize()
    held = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 20, 3 << 20, 6 << 20) for _ in range(8)]
    for i in range(5):
        out.zero_()
        g.replay()
        mid = cache.attend(prompt, SCALE, cu_q=cu, max_q=70)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert all((h == 0x5A).all() for h in held) and torch.isfinite(mid).all() and cache.error_bits() == 0


def test_two_captured_calls_replayed_at_once():
    cache, rng = filled([6000, 900], seed=5)
    queries = [rows(rng, 2, 8), rows(rng, 2, 8)]
    want = [cache.attend(x, SCALE).clone() for x in queries]
    graphs, outs = [], []
    for x in queries:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attend(x, SCALE))
        graphs.append((g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want)) and cache.error_bits() == 0


def test_captured_steps_advance_among_steps_that_are_not():
    """A step (append, attention) captured once: replays go on from the lengths that the last step left, whoever took it,
    and leave the same pages and results as steps that are not captured."""
    twin = [filled([130, 40], seed=6, P=32, spare=3)[0] for _ in range(2)]
    lens, cu, rng = [130, 40], offsets([1, 1]), np.random.default_rng(8)
    kv, query = rows(rng, 4, 2), rows(rng, 2, 8)
    array = twin[0].seq_lens.data_ptr()

    def step(cache):
        cache.append(kv[:2], kv[2:], cu, 1)
        return cache.attend(query, SCALE)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(twin[0])
    assert twin[0].seq_lens.tolist() == lens  # nothing has run yet
    for i, captured in enumerate([True, True, False, True, False, False, True, True]):
        kv.copy_(rows(rng, 4, 2)), query.copy_(rows(rng, 2, 8))
        if captured:
            g.replay()
        got = out if captured else step(twin[0])
        want = step(twin[1])
        torch.cuda.synchronize()
        assert twin[0].seq_lens.tolist() == [n + i + 1 for n in lens] == twin[1].seq_lens.tolist()
        assert torch.equal(got, want) and torch.equal(twin[0].pool, twin[1].pool)
    assert twin[0].seq_lens.data_ptr() == array and twin[0].error_bits() == 0 == twin[1].error_bits()


def test_captured_on_a_forked_stream():
    """Inside a capture a second stream branches off, attends, and joins; the replayed graph gives what a plain call gives."""
    cache, rng = filled([5000, 700], seed=9)
    a, b = rows(rng, 2, 8), rows(rng, 2, 8)
    want = [cache.attend(x, SCALE).clone() for x in (a, b)]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = [cache.attend(a, SCALE, stream=side), cache.attend(b, SCALE)]
        main.wait_stream(side)
        total = got[0] + got[1]
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(total, want[0] + want[1])
    assert cache.error_bits() == 0

"""Workspaces of the cache's attention: threads, graphs, growth."""
import threading

import pytest
import torch

from means_clustering_amd import kvcache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(lens, hq=8, hkv=2, D=128, p=16, seed=0):
    """Random cache and queries of requests with (slots in the cache, new tokens)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-s // p) for s, _ in lens]
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=g).to(torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(sum(need), p, hkv, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(sum(n for _, n in lens), hq, D, generator=g).bfloat16().to(DEV)
    start = torch.tensor([0] + [n for _, n in lens]).cumsum(0).to(torch.int32).to(DEV)
    return dict(q=q, k_cache=k, v_cache=v, block_table=table.to(DEV), query_start=start,
                seq_lens=torch.tensor([s for s, _ in lens], dtype=torch.int32, device=DEV),
                max_new=max(n for _, n in lens))


SHAPES = [[(5000, 1), (300, 1)], [(3000, 1), (200, 60), (900, 33)], [(4000, 100)], [(700, 3)] * 9]


class _Recorder:
    """Stands for the library: two calls meet, their workspaces are noted, and nothing is launched."""

    def __init__(self, real):
        self.real, self.meet, self.seen = real, threading.Barrier(2, timeout=60), []

    def __getattr__(self, name):
        return getattr(self.real, name)

    def kmeans_kv_attend(self, *args):
        ws, nbytes = args[-3], args[-2]
        if not ws:
            return kvcache.KM_ERR_WORKSPACE
        self.meet.wait()
        self.seen.append((ws, nbytes))
        self.meet.wait()
        return 0


def test_calls_of_two_threads_have_workspaces_of_their_own(monkeypatch):
    d = _inputs(SHAPES[0])
    rec = _Recorder(kvcache.lib())
    monkeypatch.setattr(kvcache, "lib", lambda: rec)
    threads = [threading.Thread(target=lambda: kvcache.attend(**d)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a, na), (b, nb) = sorted(rec.seen)
    assert a + na <= b


def test_two_threads_on_the_default_stream_equal_serial_calls():
    data = [_inputs(s, seed=i) for i, s in enumerate(SHAPES)]
    want = [kvcache.attend(**d, lse=True) for d in data]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(who):
        try:
            for i in range(40):
                j = (i * (who + 1) + who) % len(data)
                got[who, i] = j, kvcache.attend(**data[j], lse=True)
        except Exception as e:  # (a thread's exception would be lost)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(w,)) for w in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and len(got) == 80
    for j, (out, lse) in got.values():
        assert torch.equal(out, want[j][0]) and torch.equal(lse, want[j][1])


def _capture(stream, d, **kw):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = kvcache.attend(**d, lse=True, **kw)
    return graph, got


def _fill(n=24):
    """Memory of many sizes, as a program would take it next."""
    return [torch.full((1 << (10 + i % 12),), 7, dtype=torch.int32, device=DEV) for i in range(n)]


def test_graph_without_a_workspace_outlives_larger_calls():
    """An eager step, the same step captured, a larger eager step on that stream, other tensors: each replay gives the
    eager result and writes nobody else's memory."""
    small, large = _inputs(SHAPES[0]), _inputs(SHAPES[2], seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want, wl = kvcache.attend(**small, lse=True)
        want_large, _ = kvcache.attend(**large, lse=True)
    s.synchronize()
    graph, (got, gl) = _capture(s, small)
    other, (got2, _) = _capture(s, large)
    with torch.cuda.stream(s):
        kvcache.attend(**large)
    s.synchronize()
    filled = _fill()
    torch.cuda.synchronize()
    for _ in range(3):
        got.zero_(), gl.zero_(), got2.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gl, wl)
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(got2, want_large)
        kvcache.attend(**large)
        torch.cuda.synchronize()
        assert all(bool((f == 7).all()) for f in filled)


def test_graph_with_a_workspace_that_grows_later():
    """The captured buffer stays with the Workspace: memory taken after a larger call is not the graph's."""
    small, large = _inputs(SHAPES[0]), _inputs(SHAPES[2], seed=3)
    ws = kvcache.Workspace(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want, wl = kvcache.attend(**small, lse=True, ws=ws)
    s.synchronize()
    first = ws.buf.data_ptr()
    graph, (got, gl) = _capture(s, small, ws=ws)
    assert [b.data_ptr() for b in ws.captured] == [first]
    with torch.cuda.stream(s):
        want_large, _ = kvcache.attend(**large, lse=True, ws=ws)
    s.synchronize()
    assert ws.buf.data_ptr() != first and [b.data_ptr() for b in ws.captured] == [first]
    filled = _fill()
    torch.cuda.synchronize()
    for _ in range(3):
        got.zero_(), gl.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gl, wl)
        assert torch.equal(kvcache.attend(**large, ws=ws), want_large)
        torch.cuda.synchronize()
        assert all(bool((f == 7).all()) for f in filled)


def test_buffer_replaced_on_another_stream_is_not_reused_at_once():
    """A workspace allocated on one stream and outgrown on another: work in flight on that one still has the buffer."""
    n = 3 << 20
    ws = kvcache.Workspace(DEV)
    first = ws.get(n, DEV).data_ptr()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        ws.buf.zero_()
        ws.get(2 * n, DEV)
        busy = not s.query()
    again = torch.empty(n, dtype=torch.uint8, device=DEV)
    still = busy and not s.query()
    s.synchronize()
    if not still:
        pytest.skip("the stream was done too early to tell")
    assert again.data_ptr() != first


def test_workspace_that_grows_inside_a_capture():
    """A larger call captured with a workspace of an eager, smaller one; eager calls of both sizes between replays."""
    small, large = _inputs(SHAPES[0]), _inputs(SHAPES[2], seed=3)
    ws = kvcache.Workspace(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want_small = kvcache.attend(**small, ws=ws)
        want, wl = kvcache.attend(**large, lse=True)
    s.synchronize()
    graph, (got, gl) = _capture(s, large, ws=ws)
    filled = _fill()
    torch.cuda.synchronize()
    for _ in range(3):
        got.zero_(), gl.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gl, wl)
        assert torch.equal(kvcache.attend(**small, ws=ws), want_small)
        assert torch.equal(kvcache.attend(**large, ws=ws), want)
        torch.cuda.synchronize()
        assert all(bool((f == 7).all()) for f in filled)

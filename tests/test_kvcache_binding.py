"""Host-side rules of the cache binding that need no GPU."""
import weakref

import pytest
import torch

from means_clustering_amd import kvcache

from .test_kvcache_abi import FAKE, _append, _attend, _cache, _said, _tables

HOST = -1  # the device index of host tensors


def test_block_table_rows_that_overlap_are_refused():
    """A table shared by all requests as an expanded view has a row stride of 0: its rows do not lie `width` apart, and
    reading them so would leave the buffer."""
    shared = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="overlap"):
        kvcache._table(shared.expand(3, 8), HOST)
    with pytest.raises(ValueError, match="overlap"):
        kvcache._table(shared.as_strided((3, 4), (2, 1)), HOST)


def test_block_table_strides():
    big = torch.zeros(5, 12, dtype=torch.int32)
    assert kvcache._table(big[:, :7], HOST) == (5, 7, 12)
    assert kvcache._table(big[::2, :7], HOST) == (3, 7, 24)
    assert kvcache._table(big[:, :0], HOST) == (5, 0, 12)
    assert kvcache._table(big[:, 3:4], HOST) == (5, 1, 12)
    # one row, or none: nothing lies a stride apart
    assert kvcache._table(torch.zeros(8, dtype=torch.int32).as_strided((1, 8), (0, 1)), HOST) == (1, 8, 8)
    assert kvcache._table(big[:0], HOST)[:2] == (0, 12)
    with pytest.raises(ValueError, match="contiguous"):
        kvcache._table(big.t(), HOST)


def test_workspace_keeps_held_buffers():
    """A buffer whose address a graph holds outlives the growth of its Workspace; others are freed."""
    ws = kvcache.Workspace("cpu")
    first = weakref.ref(ws.get(1000, "cpu"))
    ws.hold(), ws.hold()
    second = weakref.ref(ws.get(2000, "cpu"))
    ws.get(3000, "cpu")
    assert first() is not None and second() is None and len(ws.captured) == 1
    assert ws.buf.numel() == 3000
    del ws
    assert first() is None


def test_scale_that_overflows_in_units_of_log_2():
    L = kvcache.lib()
    assert _attend(L, scale=3e38) == 1 and "scale" in _said(L)
    assert _attend(L, scale=-3e38) == 1
    assert _attend(L, scale=3e38, lw=FAKE, ws=None, nb=0) == 3  # (natural with weights; the workspace lacks)


def test_tensors_that_require_gradients_are_refused():
    """There is no backward pass, so results would have no history."""
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    x, w = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(64)
    i = torch.zeros(1, dtype=torch.int32)
    g = lambda t: t.clone().requires_grad_()
    for kw in (dict(q=g(x)), dict(k=g(x)), dict(v=g(x)), dict(k_cache=g(c)), dict(v_cache=g(c)), dict(q_weight=g(w)),
               dict(k_weight=g(w)), dict(rope=g(w)), dict(out=g(x))):
        a = dict(dict(q=x, k=x, v=x, k_cache=c, v_cache=c, slots=None), **kw)
        with pytest.raises(ValueError, match="no backward"):
            kvcache.append(**a)
        with torch.no_grad(), pytest.raises(ValueError, match="device"):  # (the next check: host tensors)
            kvcache.append(**a)
    for kw in (dict(q=g(x)), dict(k_cache=g(c)), dict(v_cache=g(c)), dict(log_weight=g(w)), dict(out=g(x)),
               dict(lse=g(w))):
        a = dict(dict(q=x, k_cache=c, v_cache=c, block_table=i[None], query_start=i, seq_lens=i), **kw)
        with pytest.raises(ValueError, match="no backward"):
            kvcache.attend(**a)
        with torch.inference_mode(), pytest.raises(ValueError, match="device"):
            kvcache.attend(**a)


def test_append_of_more_rows_than_a_launch_has():
    """Rows of more than 128 elements take 16 threads each: 2^28 of them would be a launch of 2^32 threads."""
    L = kvcache.lib()
    wide = _cache(dim=256, heads=1)
    assert _append(L, wide, T=1 << 26, hq=2) == 2 and "2^28 - 16" in _said(L)


def test_attend_of_more_query_heads_than_the_join_takes():
    L = kvcache.lib()
    wide = _cache(dim=256, heads=2)
    assert _attend(L, wide, hq=1 << 18) == 1 and "2^17" in _said(L)
    assert L.kmeans_kv_attend_workspace(wide, 4, 1 << 18, 2, 4) == 0
    assert L.kmeans_kv_attend_workspace(wide, 4, 1 << 17, 2, 4) > 0


def test_tables_in_place_are_refused():
    """Lengths that are updated while other workgroups still read them would be a race."""
    L = kvcache.lib()
    names = ("ctx", "new", "off", "free", "seq", "qs", "ps", "pos", "slots")
    apart = {name: FAKE + 256 * i for i, name in enumerate(names)}
    for out in ("seq", "qs", "ps", "pos", "slots"):
        for given in ("ctx", "new", "off", "free"):
            assert _tables(L, **dict(apart, **{out: apart[given]})) == 1 and "must not be an input" in _said(L)


def test_launches_go_to_the_device_of_the_tensors(monkeypatch):
    """A stream handle of 0 is the default stream of whichever device is current."""
    current = [0]

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *e):
            current[0] = self.before

    monkeypatch.setattr(kvcache, "_device", lambda: current[0])
    monkeypatch.setattr(kvcache.torch.cuda, "device", device)
    assert kvcache._on(1, lambda x: (x, current[0]))(7) == (7, 1)
    assert kvcache._on(0, lambda x: (x, current[0]))(8) == (8, 0)
    assert current == [0]

"""examples/compressed_cache.py: decode steps over an exact and a K-Means-compressed cache."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("compressed_cache", os.path.join(ROOT, "examples",
                                                                                   "compressed_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_equal_keys_compress_without_loss():
    """Where the prompt's keys are copies of 32 vectors, 32 centroids with their counts give the exact attention: a
    centroid is one of the vectors, its value the mean of theirs.  The compressed outputs are softmax averages of
    means rounded to bf16 (2^-8 of each), the exact ones of the values themselves; both round their softmax terms and
    results (2^-8 each), so they differ by at most 5 * 2^-8 of the largest value."""
    m = _example()
    hq, h, d, p, n = 8, 2, 64, 16, 320
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(n + 40, hq + 2 * h, d, generator=g)
    # the first slots hold one copy of each, where the centroids start: every tenth token is a new vector
    which = torch.randint(32, (n,), generator=g)
    which[::10] = torch.arange(32)
    qkv[:n, hq:hq + h] = torch.randn(32, h, d, generator=g)[which]
    qkv = qkv.to(torch.bfloat16).to("cuda:0")
    exact, short = (m.Server(hq, h, d, p, 40, 400) for _ in range(2))
    for s in (exact, short):
        s.step(qkv[:n], rotate=False)
        s.step(qkv[n:n + 20], rotate=False)
    short.compress(n, 32)
    assert int(exact.held) == 340 and int(short.held) == 52 and int(short.offset) == 288
    assert torch.isfinite(short.log_weight[short.table[0, :2].long()]).all()
    for i in range(20, 40):
        a, b = (s.step(qkv[n + i:n + i + 1], rotate=False).float() for s in (exact, short))
        assert float((a - b).abs().max()) <= 5 * 2.0 ** -8 * float(qkv[:, hq + h:].abs().max())
    assert int(short.held) == 72


def test_rotated_steps_agree_before_compression_and_stay_close_after():
    m = _example()
    hq, h, d, p, n = 8, 2, 64, 16, 512
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(n + 4, hq + 2 * h, d, generator=g).to(torch.bfloat16).to("cuda:0")
    a, b = (m.Server(hq, h, d, p, 60, 600) for _ in range(2))
    whole = a.step(qkv[:n])
    parts = torch.cat([b.step(qkv[i:min(i + 100, n)]) for i in range(0, n, 100)])  # the same prompt in chunks
    assert float((whole.float() - parts.float()).abs().max()) <= 3 * 2.0 ** -8 * float(qkv.float().abs().max())
    b.compress(256, 128)
    x, y = a.step(qkv[n:n + 4]).float(), b.step(qkv[n:n + 4]).float()
    assert torch.isfinite(y).all() and float((x - y).norm()) < float(x.norm())

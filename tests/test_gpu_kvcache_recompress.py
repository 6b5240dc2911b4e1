"""examples/compressed_cache.py: a cache that is compressed again as it grows."""
import pytest
import torch

from .test_gpu_kvcache_example import _example

pytestmark = pytest.mark.gpu


def test_compressing_twice_without_loss():
    """Two stretches of 320 tokens whose keys are copies of 32 vectors each, compressed one after the other, and tokens
    in the pages that came free: the bound is that of one compression, 5 * 2^-8 of the largest value (means, terms and
    results rounded to bf16 on one side, terms and results on the other)."""
    m = _example()
    hq, h, d, p, n = 8, 2, 64, 16, 320
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(2 * n + 60, hq + 2 * h, d, generator=g)
    for at in (0, n):
        which = torch.randint(32, (n,), generator=g)
        which[::10] = torch.arange(32)  # (where the centroids start)
        qkv[at:at + n, hq:hq + h] = torch.randn(32, h, d, generator=g)[which]
    qkv = qkv.to(torch.bfloat16).to("cuda:0")
    exact, short = (m.Server(hq, h, d, p, 46, 800) for _ in range(2))
    for s in (exact, short):
        s.step(qkv[:n], rotate=False)
        s.step(qkv[n:2 * n], rotate=False)
    freed = set(short.table[0, 2:20].tolist())
    bound = 5 * 2.0 ** -8 * float(qkv[:, hq + h:].abs().max())

    def same(first, last):
        for i in range(first, last):
            a, b = (s.step(qkv[i:i + 1], rotate=False).float() for s in (exact, short))
            assert float((a - b).abs().max()) <= bound, i

    short.compress(n, 32)
    assert int(short.held) == 32 + n and short.centroids == 32
    same(2 * n, 2 * n + 20)
    short.compress(n, 32)
    assert int(short.held) == 64 + 20 and short.centroids == 64 and int(short.offset) == 2 * (n - 32)
    same(2 * n + 20, 2 * n + 60)
    used = set(short.table[0, 4:int(short.held) // p].tolist())
    assert used & freed  # tokens lie in pages that the first compression gave back


def test_compressing_more_than_is_held_is_refused():
    m = _example()
    s = m.Server(4, 2, 64, 16, 20, 300)
    qkv = torch.randn(64, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to("cuda:0")
    s.step(qkv, rotate=False)
    for slots, clusters in ((80, 16), (64, 80), (24, 16), (32, 8), (32, 0)):
        with pytest.raises(ValueError):
            s.compress(slots, clusters)
    s.compress(48, 16)
    with pytest.raises(ValueError, match="holds 16 tokens"):
        s.compress(32, 16)
    assert int(s.held) == 32

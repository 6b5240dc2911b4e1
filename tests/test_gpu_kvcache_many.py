"""The cache's attention over many requests: threads that own several of them, pieces of the keys' line that run over
idle requests and into the next head, parts numbered across divided and whole requests."""
import random

import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, DEV, FP, Case

pytestmark = pytest.mark.gpu


def _lens(R, kind, seed):
    """(slots in the cache, new tokens): short contexts, three long ones, idle runs longer than a wavefront."""
    r = random.Random(seed)
    lens = []
    for i in range(R):
        c = int(r.choice([r.randint(0, 40), r.randint(0, 200)]))
        n = 1
        if kind != "decode" and r.random() < 0.08:
            n = r.randint(2, 70)
        lens.append((c + n, n))
    for at, c in ((R // 5, 3000), (R // 2 + 3, 5000), (R - 1, 1700)):
        lens[at] = (c, lens[at][1])
    for first, count in ((0, 3), (R // 4, 70), (R // 2 + 4, min(R // 5, 140)), (R - 12, 10)):
        for i in range(first, min(first + count, R - 1)):
            lens[i] = (r.choice([0, 33]), 0)
    if kind == "chunks":  # long prompts beside short ones, divided and whole
        lens[R // 5] = (2500, 90)
        lens[R // 2 + 3] = (1900, 130)
    return lens


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("R,hq,hkv,D,dt,p", [(65, 6, 3, 64, BF, 16), (256, 4, 4, 128, FP, 32), (257, 6, 3, 64, BF, 16),
                                             (513, 8, 2, 128, BF, 64), (1100, 3, 3, 64, FP, 16),
                                             (1100, 4, 1, 80, BF, 16)])
def test_decode_of_many_requests(R, hq, hkv, D, dt, p, window):
    Case(_lens(R, "decode", R), hq, hkv, D, dt, p, window, seed=R).check()


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("R,hq,hkv,D,dt,p", [(65, 6, 3, 64, BF, 16), (257, 6, 3, 64, FP, 16), (513, 8, 2, 128, BF, 64),
                                             (1100, 2, 2, 64, BF, 16)])
def test_mixed_steps_of_many_requests(R, hq, hkv, D, dt, p, window):
    Case(_lens(R, "mixed", R), hq, hkv, D, dt, p, window, seed=R).check()


@pytest.mark.parametrize("R,hq,hkv", [(257, 17, 1), (600, 40, 2)])
def test_one_launch_of_chunks_for_many_requests(R, hq, hkv):
    """More than 16 query heads a cache head: the chunk launch serves single tokens too."""
    Case(_lens(R, "chunks", R), hq, hkv, 64, BF, seed=R).check()


@pytest.mark.parametrize("R", [257, 1100])
def test_weighted_steps_of_many_requests(R):
    Case(_lens(R, "chunks", R), 4, 2, 64, BF, weighted=True, seed=R).check()


def test_one_busy_request_among_many():
    """The only request with tokens stands far from both ends, before and after long idle runs."""
    for at in (0, 200, 700, 1099):
        lens = [(20, 0)] * 1100
        lens[at] = (2000, 1)
        Case(lens, 4, 4, 64, BF).check()
    lens = [(0, 0)] * 900
    lens[77], lens[640] = (700, 1), (1500, 60)
    Case(lens, 4, 2, 64, BF).check()


def test_overlapping_requests_with_more_tiles_than_32_bits_count():
    """33,000 requests that all claim the same 2^19 tokens (an error of the caller): 2^31 tiles and more.  The call
    stays inside every buffer, and later calls are right."""
    T, n = 1 << 19, 33000
    q = torch.zeros(T, 16, 16, dtype=BF, device=DEV)
    k = torch.zeros(1, 16, 1, 16, dtype=BF, device=DEV)
    starts = torch.zeros(2 * n + 1, dtype=torch.int32)
    starts[1::2] = T
    out = torch.zeros_like(q)
    kvcache.attend(q, k, k, torch.zeros(2 * n, 1, dtype=torch.int32, device=DEV), starts.to(DEV),
                   torch.full((2 * n,), 16, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert bool((out == 0).all())  # (values of zero)
    Case([(300, 40), (200, 1)], 4, 2, 64, BF).check()

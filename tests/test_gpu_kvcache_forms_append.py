"""The append into an 8-bit cache where workgroups share blocks, and the paths that large calls take.  References and
bounds as in test_gpu_kvcache_forms.py."""
import math

import numpy as np
import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, DEV, FP, _rope
from .test_gpu_kvcache_forms import F8, _check_append8, _check_block_rows, _random_cache, _turned

pytestmark = pytest.mark.gpu


def _border_pairs(n, seed):
    """(p, r, cos, sin) with p cos - r sin beside 448, on different sides of it as its products are fused: the first of
    448's binade where a scale of 1 no longer holds it."""
    rng = np.random.default_rng(seed)
    f32 = lambda x: x.astype(np.float32).astype(np.float64)
    bf = lambda x: torch.from_numpy(x).to(BF).double().numpy()
    out = []
    while sum(len(o) for o in out) < n:
        p, r = bf(rng.uniform(300, 900, 4096)), bf(rng.uniform(-900, 900, 4096))
        s = f32(rng.uniform(-0.3, 0.3, 4096))
        c = f32((448 + r * s) / p)
        first, second, neither = f32(p * c - f32(r * s)), f32(f32(p * c) - r * s), f32(f32(p * c) - f32(r * s))
        keep = ((first > 448) != (second > 448)) | ((first > 448) != (neither > 448))
        out.append(np.stack([p, r, c, s], 1)[keep])
    return torch.from_numpy(np.concatenate(out)[:n])


@pytest.mark.parametrize("D,heads", [(128, 1), (256, 2), (64, 1)])
@pytest.mark.parametrize("pairs", [False, True])
def test_blocks_of_two_windows_agree_on_their_scale(D, heads, pairs):
    """Blocks of 16 slots that lie across the workgroups' windows of tokens, the largest element of each on the border of
    two scales: all of its codes are of the scale that stands there."""
    T, rot = 16 * 40, 16
    at = _border_pairs(T // 16, D)
    g = torch.Generator().manual_seed(D)
    k = (torch.rand(T, heads, D, generator=g) * 400 - 200).to(BF)
    rope = torch.cat([torch.ones(T, rot // 2), torch.zeros(T, rot // 2)], 1)
    slots = torch.arange(T, dtype=torch.int32) + 8  # (windows start at the middle of blocks)
    for b in range(T // 16):
        t = 16 * b + 8 + int(torch.randint(16, (1,), generator=g)) if b < T // 16 - 1 else T - 1
        k[t, :, 0], k[t, :, 1 if pairs else rot // 2] = float(at[b, 0]), float(at[b, 1])
        rope[t, 0], rope[t, rot // 2] = float(at[b, 2]), float(at[b, 3])
    codes, scale = _random_cache(T // 16 + 1, 16, heads, D, g)
    scale[:] = 100
    kc, ks = codes.to(DEV).view(F8), scale.to(DEV)
    pos = torch.arange(T, dtype=torch.int32)
    kvcache.append(None, k.to(DEV), None, kc, None, slots.to(DEV), positions=pos.to(DEV), rope=rope.to(DEV),
                   interleaved=pairs, k_scale=ks)
    y, mag = _turned(k, None, rope, pos[None].long(), torch.zeros(rot // 2, dtype=torch.long), 0.0, pairs)
    assert float((y.abs().amax((1, 2)) > 440).sum()) >= T // 16
    _check_block_rows(codes, scale, kc.view(torch.uint8).cpu(), ks.cpu(), slots, [True] * T, y, mag, D)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_queries_are_the_same_in_every_call(dt, pairs, norm):
    """A query's row is the same to the last bit beside a 16-bit cache, beside an 8-bit one, and in a large call, whose
    queries have a launch of their own."""
    T, hq, D = 4200, 32, 128
    g = torch.Generator().manual_seed(7)
    q = torch.randn(T, hq, D, generator=g).to(dt).to(DEV)
    k = torch.randn(T, 1, D, generator=g).to(dt).to(DEV)
    pos = torch.randint(0, 400, (T,), generator=g, dtype=torch.int32).to(DEV)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(DEV) if norm else None
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    kw = dict(rope=_rope(400, D).to(DEV), q_weight=w, k_weight=w, interleaved=pairs)
    pages = -(-T // 16)
    plain = kvcache.append(q, k, None, torch.zeros(pages, 16, 1, D, dtype=dt, device=DEV), None, slots, positions=pos,
                           **kw)
    kc = torch.zeros(pages, 16, 1, D, dtype=torch.uint8, device=DEV).view(F8)
    ks = torch.zeros(pages, 1, 1, dtype=torch.uint8, device=DEV)
    large = kvcache.append(q, k, None, kc, None, slots, positions=pos, k_scale=ks, **kw)
    codes, scale = kc.view(torch.uint8).clone(), ks.clone()
    small = torch.cat([kvcache.append(q[i:i + 600], k[i:i + 600], None, kc, None, slots[i:i + 600],
                                      positions=pos[i:i + 600], k_scale=ks, **kw) for i in range(0, T, 600)])
    assert torch.equal(plain, large) and torch.equal(plain, small)
    whole = (torch.arange(T) // 600 == (torch.arange(T) // 16 * 16) // 600) & (
        torch.arange(T) // 600 == (torch.arange(T) // 16 * 16 + 15).clamp(max=T - 1) // 600)
    whole = whole.to(DEV)  # slots of blocks that one of the small calls writes as a whole
    assert torch.equal(codes.view(-1, D)[:T][whole], kc.view(torch.uint8).view(-1, D)[:T][whole])
    assert torch.equal(scale.view(-1).repeat_interleave(16)[:T][whole], ks.view(-1).repeat_interleave(16)[:T][whole])


def _ragged(T, short=40):
    """A long run in the middle of a block, short ones (decode steps and a few tokens) and a second long one."""
    runs = [(i % 16, 1 + i % 3) for i in range(short)]
    left = T - sum(n for _, n in runs)
    return [(5, left * 2 // 3)] + runs + [(11, left - left * 2 // 3)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,hq,hkv,D,rot,pairs,norm,layout,axes,values", [
    (5500, 13, 3, 256, 256, False, True, "packed", None, True),   # odd heads, the last workgroup has one; queries apart
    (5500, 1, 3, 256, 128, True, True, "plain", 3, False),        # keys alone
    (6700, 0, 5, 128, 128, False, True, "packed", None, True),
    (8300, 4, 4, 128, 96, True, False, "heads", 2, True),
    (2100, 32, 8, 256, 256, False, False, "packed", 3, True),
    (9400, 1, 7, 48, 32, False, True, "packed", 4, False)])
def test_large_appends(dt, T, hq, hkv, D, rot, pairs, norm, layout, axes, values):
    """Workgroups of two heads: where windows of 4,096 / lanes tokens times heads reach 1,024; from 65,536 rows of D =
    256 (131,072 of 128) on the queries have a launch of their own."""
    lanes = next(n for n in (2, 4, 8, 16) if 16 * n >= D)
    assert -(-T * lanes // 256) * hkv >= 1024
    _check_append8(_ragged(T), hq, hkv, D, 16, dt, rot, pairs, norm, layout, axes, padding=True, seed=T, values=values)


def test_large_appends_of_few_heads():
    """One head a workgroup, and windows of which the last has few tokens."""
    _check_append8(_ragged(8209), 9, 1, 128, 64, BF, seed=1)
    _check_append8(_ragged(4097), 17, 2, 256, 32, FP, rot=64, axes=3, mix=0, seed=2)

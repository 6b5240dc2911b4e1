"""What a row of the attention's further forms does not see never reaches it, to the last bit; scores at the ends of
fp32.  References and bounds as in test_gpu_kvcache_forms.py."""
import math

import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, DEV, FP
from .test_gpu_kvcache_forms import FormCase

pytestmark = pytest.mark.gpu


def _bits(got):
    out, lse = got
    return out.view(torch.int16).cpu(), lse.view(torch.int32).cpu()


def _attend(c):
    return _bits(kvcache.attend(**c.device(), lse=True))


def _same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _free_page_0(c):
    """Gives page 0, which stands for pages that are not held where a load needs one, to nobody."""
    held = set(int(x) for x in c.table.flatten() if x >= 0)
    if 0 not in held:
        return
    other = next(i for i in range(c.k.shape[0]) if i not in held)
    c.table[c.table == 0] = other
    arrays = [c.k, c.v] + ([] if c.lw is None else [c.lw]) + ([t for p in c.codes for t in p] if c.eight else [])
    for t in arrays:
        t[[0, other]] = t[[other, 0]]


def _fill_unseen(c, key, code):
    """Keys (and codes) of everything that no query sees: slots behind the sequences, pages of nobody, slots that their
    weight removes, slots in front of the windows."""
    p, held = c.p, torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for r, (s, n) in enumerate(c.lens):
        lo = max(0, s - n - c.window + 1) if c.window else 0
        for j in range(s):
            seen = j >= lo or (c.prefix is not None and j < c.prefix[r])
            page = int(c.table[r, j // p])
            if seen and 0 <= page < c.k.shape[0] and (c.lw is None or float(c.lw[page, 0, j % p]) > -math.inf):
                held[page, j % p] = True
    c.k[~held] = key
    c.v[~held] = 1.0
    if c.eight:
        for codes, _ in c.codes:
            codes[~held] = code


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("n,hq", [(1, 8), (5, 4), (90, 4)])
@pytest.mark.parametrize("eight,cap,sharp", [(False, 2.0, 0.3), (False, 30.0, 1.0), (False, 44.0, 0.2),
                                             (False, 200.0, 1.0), (True, 1.0, 0.2)])
@pytest.mark.parametrize("window,prefix,weighted", [(0, None, False), (40, [20, 3], False), (50, None, True)])
def test_capped_rows_do_not_depend_on_what_they_do_not_see(dt, n, hq, eight, cap, sharp, window, prefix, weighted):
    make = lambda: FormCase([(150, n), (100, n)], hq, 2, 64, dt, window=window, eight=eight, prefix=prefix, cap=cap,
                            sharp=sharp, weighted=weighted)
    got = []
    for key, code in ((0.01, 0), (1e4, 0x7e)):
        c = make()
        if weighted:  # (one weight for all heads of a slot)
            c.lw[:] = c.lw[:, :1]
        _free_page_0(c)
        c.table[0, 2] = -1
        _fill_unseen(c, key, code)
        got.append(_attend(c))
    assert _same(*got)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n", [1, 4, 90])
@pytest.mark.parametrize("cap", [1.0, 20.0, 100.0])
def test_capped_rows_do_not_depend_on_other_rows(n, cap, eight):
    """One head's and one token's queries a thousand times as large: the others' results stay as they are."""
    c = FormCase([(150, n), (100, n)], 8, 2, 64, BF, cap=cap, sharp=0.1, eight=eight)
    small = _attend(c)
    c.q[:, 2] *= 1000
    c.q[n // 2] *= 1000
    large = _attend(c)
    keep = torch.ones(2 * n, 8, dtype=torch.bool)
    keep[:, 2] = keep[n // 2] = False
    assert torch.equal(small[0][keep], large[0][keep]) and torch.equal(small[1][keep], large[1][keep])
    assert not torch.equal(small[0][:, 2], large[0][:, 2])


def _one_key_scores(cap, x, chunk, weighted=False, scale=1.0, slopes=None):
    """lse (and results) of rows that see one key each, whose products are x: with one key lse is the score."""
    n = len(x)
    c = FormCase([(n, n)] if chunk else [(1, 1)] * n, 2, 1, 64, BF, window=1, cap=cap, weighted=weighted)
    c.q[:], c.scale = 0, scale
    c.q[:, :, 0] = 1.0
    for i in range(n):
        key = torch.zeros(64)
        key[0] = x[i]
        c.set(0 if chunk else i, i if chunk else 0, k=key.to(BF), lw=0.0 if weighted else None)
    d = c.device()
    if slopes is not None:
        d["slopes"] = slopes
    out, lse = kvcache.attend(**d, lse=True)
    v = torch.stack([c.v[int(c.table[0, i // c.p]), i % c.p, 0] if chunk else c.v[int(c.table[i, 0]), 0, 0]
                     for i in range(n)])
    assert torch.equal(out.cpu(), v[:, None].expand(n, 2, 64))
    return lse.double().cpu()


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("cap", [1.0, 30.0, 44.0, 50.0, 64.0, 64.5, 90.0, 95.0, 1000.0])
def test_capped_score_of_one_key(cap, weighted, chunk):
    """With t = tanh y and e = 2^-24: the formula of caps up to 64 is off by 4 e cap, below zero by 5 e |t| cap more; of
    y itself three roundings (scale / cap, its factor, the product) are 3 e |y| (1 - t^2) <= 1.4 e cap.  Beyond 64 both
    are parts of the score: 6 e of it and, |y| (1 - t^2) <= |t|, 3 e.  Then the cap in its unit, log 2 and the products
    with them: 4 e of the score."""
    y = torch.tensor([0.001, 0.01, 0.1, 0.3, 0.5, 0.62, 0.63, 0.7, 1.0, 1.5, 2.0, 3.0, 5.0, 9.0, 30.0])
    x = (torch.cat([y, -y, torch.zeros(1)]) * cap).to(BF)
    lse = _one_key_scores(cap, x, chunk, weighted)
    t = torch.tanh(x.double() / cap)
    e, s = 2.0 ** -24, (cap * t).abs()
    tol = (5.4 + 5 * (t < 0) * t.abs()) * e * cap + 4 * e * s if cap <= 64 else 13 * e * s
    off = (lse - (cap * t)[:, None]).abs() - tol[:, None]
    assert float(off.max()) <= 0, off


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_caps_near_the_end_of_fp32(weighted, chunk):
    """Twice the cap is no float; the score is, as near as beyond a cap of 64."""
    cap, scale = 2e38, 4.0
    y = torch.tensor([0.1, 0.6, 0.7, 1.0, 2.0, 5.0])
    k = (torch.cat([y, -y, torch.zeros(1)]) * (cap / scale)).to(BF)
    lse = _one_key_scores(cap, k, chunk, weighted, scale=scale)
    s = cap * torch.tanh(k.double() * (scale / cap))
    assert bool(((lse - s[:, None]).abs() <= 13 * 2.0 ** -24 * s.abs()[:, None]).all()), lse


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_slopes_near_the_end_of_fp32(weighted, chunk):
    """At distance 0 a finite slope takes nothing, even where times log2(e) it is no float; beyond, nothing is left."""
    slopes = torch.tensor([3e38, 2.5e38], device=DEV)
    x = torch.tensor([0.0, 1.0, -3.0, 0.5])
    lse = _one_key_scores(0.0, x, chunk, weighted, slopes=slopes)
    assert float((lse - x.double()[:, None]).abs().max()) <= 8 * 2.0 ** -24 * 3
    n = 70 if chunk else 1
    c = FormCase([(100, n)], 2, 1, 64, BF, weighted=weighted)
    if weighted:
        c.lw.zero_()
    out = kvcache.attend(**dict(c.device(), slopes=slopes)).cpu()
    own = torch.stack([c.v[int(c.table[0, j // 16]), j % 16, 0] for j in range(100 - n, 100)])
    assert torch.equal(out, own[:, None].expand(n, 2, 64))


@pytest.mark.parametrize("what", ["key", "value", "key scale", "value scale"])
@pytest.mark.parametrize("dt,n,hq,D", [(BF, 1, 8, 64), (FP, 4, 4, 128), (BF, 90, 4, 64), (FP, 70, 2, 80), (BF, 1, 4, 256),
                                       (BF, 60, 2, 256)])
@pytest.mark.parametrize("window,prefix,weighted,cap", [(0, None, False, 0.0), (40, None, True, 0.0),
                                                        (40, [30, 60], False, 5.0)])
def test_unseen_nan_codes_and_scales_do_not_reach_a_row(what, dt, n, hq, D, window, prefix, weighted, cap):
    """NaN codes of a slot, or a scale of 255 for a block's 16 slots: rows that see one of them are NaN, all others have
    the bits that they have without."""
    bad = {0: [149, 100, 2], 1: [99, 50, 20]}  # slots; of a scale their blocks
    make = lambda: FormCase([(150, n), (100, n)], hq, 2, D, dt, window=window, eight=True, prefix=prefix,
                            weighted=weighted, cap=cap)
    clean = make()
    want = kvcache.attend(**clean.device()).cpu()
    for r, js in bad.items():
        for j in js:
            c = make()
            page = int(c.table[r, j // 16])
            codes, scale = c.codes["value" in what]
            if "scale" in what:
                scale[page] = 255
                hit = range(j - j % 16, min(j - j % 16 + 16, c.lens[r][0]))
            else:
                codes[page, j % 16] = 0xff
                hit = [j]
            got = kvcache.attend(**c.device()).cpu()
            for t in range(2 * n):
                mine, i = (t // n == r), t % n
                pos = c.lens[r][0] - n + i
                sees = torch.zeros(2, dtype=torch.bool)
                for s in hit if mine else ():
                    if (s <= pos and (not window or s > pos - window)) or (prefix and s < prefix[r]):
                        sees |= torch.ones(2, dtype=torch.bool) if c.lw is None else c.lw[page, :, s % 16] > -math.inf
                sees = sees.repeat_interleave(hq // 2)
                assert bool(got[t][sees].isnan().all()), (r, j, t)
                assert torch.equal(got[t][~sees].view(torch.int16), want[t][~sees].view(torch.int16)), (r, j, t)


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-46])
def test_caps_that_fp32_has_not(cap):
    """Rounded to 0 it would mean no cap at all."""
    d = FormCase([(20, 1)], 2, 1, 64, BF).device()
    with pytest.raises(ValueError, match="softcap"):
        kvcache.attend(**dict(d, softcap=cap))
    kvcache.attend(**dict(d, softcap=0.0))
    kvcache.attend(**dict(d, softcap=0))

"""Edges of the cache's operators: page numbers, lengths, windows, scales and terms at the ends of their ranges."""
import math

import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, DEV, E, FP, U, Case

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------------ tables ----

@pytest.mark.parametrize("p", [16, 64, 1 << 20])
def test_tables_pages_that_no_cache_can_have(p):
    """A page of 2^31 / page_size or more has no slot: its first slots would wrap to those of page 0."""
    last = 2 ** 31 // p - 1
    pages = [last, last + 1, 2 * last + 2, 2 ** 31 - 1, 2, -5]
    pages = [min(x, 2 ** 31 - 1) for x in pages]
    want = [x * p + 3 if 0 <= x <= last else -1 for x in pages]
    R = len(pages)
    # held pages, read from the table
    t = kvcache.tables(_i32([3] * R), _i32([1] * R), _i32(pages).view(R, 1), _i32([0]), p, R)
    assert t.slots.tolist() == want
    # new pages, from the free list
    table = torch.full((R, 1), -7, dtype=torch.int32, device=DEV)
    t = kvcache.tables(_i32([0] * R), _i32([4] * R), table, _i32(pages), p, 4 * R)
    assert t.slots.tolist()[3::4] == want
    assert table.view(-1).tolist() == pages
    # and nothing is appended for them
    if p == 16:
        cache = torch.zeros(4, p, 1, 16, dtype=BF, device=DEV)
        kvcache.append(None, torch.ones(4 * R, 1, 16, dtype=BF, device=DEV), None, cache, None, t.slots)
        assert bool((cache[2, :4] == 1).all()) and float(cache.float().sum()) == 4 * 16


def test_tables_arrays_without_elements_have_any_address():
    """No new tokens and no free pages: their arrays may begin where another one does."""
    L = kvcache.lib()
    ctx, new, table = _i32([20, 3]), _i32([0, 0]), _i32([[4, 5], [6, -1]])
    out = _i32([-9] * 8)
    at = out.data_ptr()
    status = L.kmeans_kv_tables(ctx.data_ptr(), new.data_ptr(), None, 2, 16, table.data_ptr(), 2, 2, at, 0, 0, at, at + 8,
                                at + 20, ctx.data_ptr(), new.data_ptr(), kvcache._stream(0))
    assert status == 0, L.kmeans_kv_last_error().decode()
    assert out.tolist() == [20, 3, 0, 0, 0, 0, 0, 0] and ctx.tolist() == [20, 3]


# ------------------------------------------------------------------------------------------------------ attend ----

def _check(c, **changes):
    """The call against Case.reference, its tolerances and its rule for rows that see nothing."""
    _near(c, *kvcache.attend(**dict(c.device(), **changes), lse=True))


def _near(c, out, lse):
    torch.cuda.synchronize()
    ro, rl, to, tl = c.reference()
    got, gl = out.double().cpu(), lse.double().cpu()
    assert bool(((got - ro).abs() <= to).all()), ((got - ro).abs() - to).max()
    empty = rl == -math.inf
    assert bool((gl[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
    assert bool(((gl[~empty] - rl[~empty]).abs() <= tl[~empty]).all())


@pytest.mark.parametrize("n", [1, 12, 60])
@pytest.mark.parametrize("window", [63, 64, 65, 80, 100, 5000, 2 ** 31 - 1])
def test_attend_window_over_a_row_shorter_than_its_request(n, window):
    """100 slots, of which the table row holds 64: the last query stands at slot 99 and sees those after 99 - window."""
    c = Case([(100, n), (70, 1)], 4, 2, 64, BF, window=window)
    c.table[:, 4:] = -1
    print(f"[attend] n={n} window={window}", flush=True)
    _check(c, block_table=c.table[:, :4].contiguous().to(DEV))


@pytest.mark.parametrize("last,kept", [(30, 1), (30, 15), (3, 2), (90, 40), (90, 89)])
@pytest.mark.parametrize("window", [0, 50])
def test_attend_request_cut_off_by_the_capacity(last, kept, window):
    """query_start passes T: the last request's first tokens keep their slots, and the slots of the others, which
    nobody wrote, are not read."""
    c = Case([(50, 20), (120, last)], 4, 2, 64, BF, window=window)
    ro, rl, to, tl = c.reference()
    for j in range(120 - last + kept, 120):
        c.set(1, j, k=math.nan, v=math.nan)
    d, T = c.device(), 20 + kept
    print(f"[attend] last={last} kept={kept} window={window}", flush=True)
    out, lse = kvcache.attend(**dict(d, q=d["q"][:T].contiguous(), max_new=max(20, last)), lse=True)
    assert bool(((out.double().cpu() - ro[:T]).abs() <= to[:T]).all())
    assert bool(((lse.double().cpu() - rl[:T]).abs() <= tl[:T]).all())


def test_step_with_more_tokens_than_the_capacity():
    """tables, append and attend with `total` below the sum of the new lengths: the tokens that have rows are answered
    as if all were there."""
    g = torch.Generator().manual_seed(4)
    p, hq, h, D = 16, 4, 2, 64
    ctx, new, cap = [40, 21], [6, 50], 33
    rows = torch.randn(56, hq + 2 * h, D, generator=g).to(BF).to(DEV)
    old = torch.randn(2, 48, h, D, generator=g).to(BF).to(DEV)

    def step(total):
        k = torch.full((16, p, h, D), math.nan, dtype=BF, device=DEV)
        v = k.clone()
        table = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
        table[0, :3], table[1, :2] = _i32([1, 2, 3]), _i32([5, 6])
        for r, c in enumerate(ctx):
            at = torch.arange(c, device=DEV)
            k[table[r].long()[at // p], at % p] = v[table[r].long()[at // p], at % p] = old[r, :c]
        t = kvcache.tables(_i32(ctx), _i32(new), table, _i32(list(range(8, 16))), p, total)
        x = rows[:total]
        q = kvcache.append(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], k, v, t.slots)
        return kvcache.attend(q, k, v, table, t.query_start, t.seq_lens, lse=True)

    (whole, wl), (cut, cl) = step(56), step(cap)
    # both round the terms and the result (2^-8 each) of values of at most |v|
    most = max(float(rows[:, hq + h:].abs().max()), float(old.abs().max()))
    assert float((whole[:cap].float() - cut.float()).abs().max()) <= 4 * 2.0 ** -8 * most
    assert float((wl[:cap] - cl).abs().max()) <= 1e-4


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dt", [BF, FP])
def test_attend_scores_of_any_size(dt, n, weighted):
    """Scores from thousands to 2^31: no term leaves the type, whatever the scores' own rounding makes of them."""
    for size in (4.0, 64.0, 512.0, 2048.0, 4096.0, 16384.0):
        c = Case([(300, n)], 4, 2, 64, dt, weighted=weighted, sharp=size)
        c.k = torch.where(torch.isnan(c.k), c.k, (c.k.float() * size).clamp(-65504, 65504).to(dt))
        c.q = (c.q.float().nan_to_num(posinf=65504.0, neginf=-65504.0)).to(dt)  # (fp16: randn beyond 4 has overflowed)
        c.scale = 1.0
        out, lse = kvcache.attend(**c.device(), lse=True)
        seen = c.v[torch.isfinite(c.v)].abs().max()
        assert bool(torch.isfinite(out).all()) and float(out.abs().max()) <= 1.01 * float(seen)
        want = c.reference()[1]
        bound = 80 * E * float(c.q.double().abs().max()) * float(c.k[torch.isfinite(c.k)].double().abs().max()) * 64
        assert bool(((lse.double().cpu() - want).abs() <= bound + 1e-4).all())


def _sink(keys, n, hkv, R, at, weighted):
    """Requests over one set of pages whose slot `at` has a score 18 (e^18 is 2^26) above the others', and a value of
    zero: the result is made of terms near 2^-26 of the largest."""
    g = torch.Generator().manual_seed(keys + n + at)
    D, p = 64, 64
    k = (0.3 * torch.randn(keys, hkv, D, generator=g)).half()
    v = (1 + 0.1 * torch.randn(keys, hkv, D, generator=g)).half()
    k[at], v[at] = 0, 0
    k[at, :, 0] = 18
    q = (0.5 * torch.randn(R * n, hkv, D, generator=g)).half()
    q[..., 0] = 8
    table = torch.arange(keys // p, dtype=torch.int32).repeat(R, 1)
    d = dict(q=q.to(DEV), k_cache=k.view(-1, p, hkv, D).to(DEV), v_cache=v.view(-1, p, hkv, D).to(DEV),
             block_table=table.to(DEV), query_start=_i32([n * r for r in range(R + 1)]), seq_lens=_i32([keys] * R),
             scale=0.125, max_new=n,
             log_weight=torch.zeros(keys // p, hkv, p, device=DEV) if weighted else None)
    sc = 0.125 * q.double().transpose(0, 1) @ k.double().permute(1, 2, 0)
    es = (D + 16) * E * 0.125 * (q.double().abs().transpose(0, 1) @ k.double().abs().permute(1, 2, 0)).amax(2)
    i = torch.arange(R * n) % n
    sc.masked_fill_(torch.arange(keys)[None, None] > (keys - n + i)[None, :, None], -math.inf)
    pr, vv = torch.softmax(sc, 2), v.double().transpose(0, 1)
    # fp16 terms hold 2^-39 of the largest; the result's own step is 2^-24 below 2^-14
    tol = (2.1 * U[FP] + 4 * es + (keys / 32 + 64) * E)[..., None] * (pr @ vv.abs()) + (
        keys * 2.0 ** -39 * float(vv.abs().max()) + 2.0 ** -25)
    lse = torch.logsumexp(sc, 2)
    ltol = es + (keys / 32 + 64) * E + 4 * E * lse.abs()
    return d, (pr @ vv).transpose(0, 1), tol.transpose(0, 1), lse.t(), ltol.t()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("keys,n,hkv,R,at", [(4096, 1, 8, 96, 0), (4096, 1, 8, 96, 4000), (4096, 20, 2, 9, 7),
                                             (16384, 256, 8, 1, 0), (16384, 256, 8, 1, 16000), (2048, 128, 4, 64, 3)])
def test_attend_fp16_terms_far_below_the_largest(keys, n, hkv, R, at, weighted):
    d, want, tol, wl, ltol = _sink(keys, n, hkv, R, at, weighted)
    print(f"[attend] keys={keys} n={n} hkv={hkv} R={R} at={at} weighted={weighted}", flush=True)
    out, lse = kvcache.attend(**d, lse=True)
    assert bool(((out.double().cpu() - want).abs() <= tol).all())
    assert bool(((lse.double().cpu() - wl).abs() <= ltol).all())


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-35, -1e-35, 1e-40, -0.125])
def test_attend_scales(scale, n, weighted):
    """Products of 2^100: a scale of 0 makes every score 0, tiny ones (a denormal too) count as they are."""
    c = Case([(150, n), (40, n if n < 40 else 40)], 4, 2, 64, BF, weighted=weighted)
    if abs(scale) < 0.1:
        c.q, c.k = (c.q.float() * 2.0 ** 50).to(BF), (c.k.float() * 2.0 ** 50).to(BF)
    c.scale = scale
    out, lse = kvcache.attend(**c.device(), lse=True)
    c.scale = abs(scale)  # (the reference takes its tolerance times the scale)
    if scale < 0:
        c.q = -c.q
    _near(c, out, lse)


@pytest.mark.parametrize("n", [1, 90])
def test_attend_scale_of_zero_with_infinite_queries(n):
    """0 times an infinite product is NaN in the row that has it, and in no other."""
    c = Case([(150, n), (40, 1)], 4, 2, 64, BF)
    c.q[0, 1, 3] = math.inf
    c.scale = 0.0
    out = kvcache.attend(**c.device())
    nan = torch.isnan(out)
    assert bool(nan[0, 1].all()) and int(nan.sum()) == 64


# ----------------------------------------------------------------------------------------------------- binding ----

def test_tensors_of_other_dimensions_are_refused():
    d = Case([(50, 1)], 4, 2, 64, BF).device()
    k = d["k_cache"][0, :1]
    for bad in (d["q"][0], d["q"][0, 0], d["q"][0, 0, 0], d["q"][None]):
        with pytest.raises(ValueError, match="q must be"):
            kvcache.attend(**dict(d, q=bad))
        with pytest.raises(ValueError, match="q must be"):
            kvcache.append(bad, k, None, d["k_cache"], None, None)
        with pytest.raises(ValueError, match="k must be"):
            kvcache.append(None, bad, None, d["k_cache"], None, None)


def test_attend_without_lse():
    d = Case([(50, 1)], 4, 2, 64, BF).device()
    want = kvcache.attend(**d)
    assert torch.equal(kvcache.attend(**d, lse=None), want) and torch.equal(kvcache.attend(**d, lse=True)[0], want)

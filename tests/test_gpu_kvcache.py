"""The paged key/value cache operators against plain 64-bit references on the CPU.

Tolerances follow from the arithmetic.  With unit roundoff u of the 16-bit type (2^-8 bf16, 2^-11 fp16) and e = 2^-24:
  append  the fp32 steps before the one rounding lose at most c e of the larger term of a rotated pair (c = D / 8 + 24
          covers the sum of squares, root, division and products), the rounding u |y|;
  attend  scores lose es = (D + 16) e scale max_j sum |q_d k_d| (+ 4 e of the weight), each softmax term its rounding u,
          the result u again: |error| <= (2.1 u + 4 es + (keys / 32 + 64) e) sum_j softmax_j |v_j|; fp16 terms below
          2^-14 lose 2^-25 absolute each.  lse: es + (keys / 32 + 64) e + 4 e |lse|.
Slots that no request holds are NaN in every test, so a read of one shows.
"""
import math
import random

import numpy as np
import pytest
import torch

from means_clustering_amd import KMeansError, kvcache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16


# ------------------------------------------------------------------------------------------------------ tables ----

def _ref_tables(ctx, new, table, free, p, total, offset):
    table = table.copy()
    qs, ps, pos, slots = [0], [0], [0] * total, [-1] * total
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        for col in range(-(-c // p), -(-(c + n) // p)):
            e = ps[-1] + col - -(-c // p)
            if col < table.shape[1]:
                table[r, col] = free[e] if e < len(free) else -1
        ps.append(ps[-1] + -(-(c + n) // p) - -(-c // p))
        for i in range(n):
            t = qs[-1] + i
            if t < total:
                pos[t] = c + i + (offset[r] if offset is not None else 0)
                col = (c + i) // p
                page = table[r, col] if col < table.shape[1] else -1
                slots[t] = page * p + (c + i) % p if page >= 0 else -1
        qs.append(qs[-1] + n)
    seq = [max(c, 0) + max(n, 0) for c, n in zip(ctx, new)]
    return table, seq, qs, ps, pos, slots


def _check_tables(ctx, new, width, p, num_free, total=None, offset=False, stride=0, seed=0):
    r = np.random.default_rng(seed)
    R = len(ctx)
    need = sum(-(-(max(c, 0) + max(n, 0)) // p) for c, n in zip(ctx, new))
    order = r.permutation(need + num_free + 7)
    table, at = r.integers(-5, -1, size=(R, width)), 0
    for i, c in enumerate(ctx):
        k = min(-(-max(c, 0) // p), width)
        table[i, :k] = order[at:at + k]
        at += k
    free = order[at:at + num_free]
    off = r.integers(0, 5000, size=R) if offset else None
    total = sum(max(n, 0) for n in new) if total is None else total
    ref = _ref_tables(ctx, new, table, free, p, total, off)
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32).reshape(-1), device=DEV)
    big = torch.full((R, width + stride), -77, dtype=torch.int32, device=DEV)
    tab = big[:, :width]
    tab.copy_(torch.from_numpy(table.astype(np.int32)))
    print(f"[tables] R={R} width={width} page={p} free={num_free} total={total}", flush=True)
    for _ in range(2):  # the call changes nothing that it reads
        t = kvcache.tables(i32(ctx), i32(new), tab, i32(free), p, total, None if off is None else i32(off))
        assert tab.cpu().tolist() == ref[0].tolist()
        for got, want in zip(t, ref[1:]):
            assert got.cpu().tolist() == [int(x) for x in want]
    assert stride == 0 or bool((big[:, width:] == -77).all())


@pytest.mark.parametrize("R,ctx,new,p", [(1, 0, 1, 16), (1, 100, 1, 16), (3, 33, 40, 32), (255, 300, 9, 16),
                                         (256, 64, 1, 64), (257, 65, 20, 16), (513, 100, 5, 128), (4096, 40, 3, 16),
                                         (4097, 40, 3, 16), (9001, 20, 2, 16)])
def test_tables(R, ctx, new, p):
    r = random.Random(R)
    c = [r.randint(0, ctx) for _ in range(R)]
    n = [r.choice([0, 1, 1, r.randint(0, new)]) for _ in range(R)]
    width = max(-(-(a + b) // p) for a, b in zip(c, n)) + 1
    _check_tables(c, n, width, p, sum(n) + 3, offset=R % 2 == 0, stride=R % 3, seed=R)


def test_tables_edges():
    _check_tables([0, 0, 0], [0, 0, 0], 2, 16, 4)                       # nothing new
    _check_tables([], [], 4, 16, 4, total=3)                            # no request, padding only
    _check_tables([5, -3, 16], [3, 4, -1], 3, 16, 4)                    # negative lengths count as 0
    _check_tables([15, 16, 17, 31], [1, 1, 1, 2], 3, 16, 4, total=9)    # page edges, padding
    _check_tables([15, 16, 17, 31], [9, 9, 99, 2], 9, 16, 3)            # the free list runs out
    _check_tables([15, 16], [0, 9], 2, 16, 0)                           # an empty free list
    _check_tables([30, 16], [40, 9], 3, 16, 9)                          # a table row runs out
    _check_tables([7, 9], [30, 50], 8, 16, 9, total=41)                 # more tokens than the capacity
    _check_tables([100], [20000], 400, 64, 400)                         # one long prompt


def test_tables_lengths_near_the_end_of_32_bits():
    """Slots that no table row can hold: nothing is written beside the table, and the tokens get no slot."""
    top = 2 ** 31 - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    big = torch.full((4, 9), -77, dtype=torch.int32, device=DEV)
    t = kvcache.tables(i32([top, top - 20, 0]), i32([5, 9, 2]), big[1:, :6], i32([3, 4, 5]), 16, 16)
    assert t.slots.tolist()[:14] == [-1] * 14
    assert t.query_start.tolist() == [0, 5, 14, 16]
    keep = big.clone()
    keep[3, 0] = -77
    assert bool((keep == -77).all())
    kvcache.tables(i32([0, 0, 0]), i32([top, top, top]), big[1:, :6], i32([3, 4, 5]), 16, 16)  # the sum wraps
    assert bool((big[0] == -77).all()) and bool((big[:, 6:] == -77).all())


# ------------------------------------------------------------------------------------------------------ append ----

def _rope(max_pos, rot):
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _ref_rows(x, w, rope, pos, eps, pairs):
    """Rows in 64 bits, and the size of the terms that each element is made of."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    mag = y.abs()
    if rope is not None:
        half = rope.shape[1] // 2
        c, s = rope[pos, None, :half].double(), rope[pos, None, half:].double()
        ia = torch.arange(half) * 2 if pairs else torch.arange(half)
        ib = ia + 1 if pairs else ia + half
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def _near_rows(got, ref, mag, dt, D):
    err = (got.double().cpu() - ref).abs()
    tol = U[dt] * ref.abs() * 1.001 + (D / 8 + 24) * E * mag + (2.0 ** -25 if dt == FP else 1e-38)
    assert bool((err <= tol).all()), (err - tol).max()


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,hq,hkv,D,rot,pairs,norm,layout", [
    (1, 8, 2, 128, 128, False, True, "packed"), (5, 4, 4, 64, 32, True, False, "plain"),
    (37, 7, 1, 80, 80, False, True, "heads"), (64, 3, 3, 256, 128, False, True, "packed"),
    (129, 2, 1, 16, 16, True, True, "plain"), (33, 5, 5, 48, 16, False, False, "heads"),
    (250, 6, 2, 112, 96, True, True, "plain"), (17, 1, 1, 240, 240, False, True, "packed"),
    (9, 4, 2, 32, 0, False, True, "plain"), (11, 4, 2, 128, 0, False, False, "plain")])
def test_append(dt, T, hq, hkv, D, rot, pairs, norm, layout):
    g = torch.Generator().manual_seed(T * D)
    p, pages, eps = 16, -(-T // 16) + 2, 1e-5
    if layout == "packed":
        x = torch.randn(T, hq + 2 * hkv, D, generator=g).to(dt)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        xd = x.to(DEV)
        qd, kd, vd = xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:]
    else:
        q, k, v = (torch.randn(T, n, D, generator=g).to(dt) for n in (hq, hkv, hkv))
        qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    shape = (pages, p, hkv, D) if layout != "heads" else (pages, hkv, p, D)
    kc0, vc0 = torch.randn(shape, generator=g).to(dt), torch.randn(shape, generator=g).to(dt)
    kc, vc = kc0.to(DEV), vc0.to(DEV)
    if layout == "heads":
        kc0, vc0, kc, vc = (t.transpose(1, 2) for t in (kc0, vc0, kc, vc))
    slots = torch.randperm(pages * p, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    if T > 8:  # padding: no slot, a slot past the cache, a position past the table
        slots[3], slots[5] = -1, pages * p
        if rot:
            pos[6] = 500
    dead = (slots < 0) | (slots >= pages * p) | ((pos >= 500) if rot else torch.zeros(T, dtype=torch.bool))
    rope = _rope(500, rot) if rot else None
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g), 1 + 0.3 * torch.randn(D, generator=g)) if norm else (None, None)
    to = lambda t: None if t is None else t.to(DEV)
    print(f"[append] T={T} hq={hq} hkv={hkv} D={D} rot={rot} {layout} {dt}", flush=True)
    out = kvcache.append(qd, kd, vd, kc, vc, to(slots), positions=to(pos) if rot else None, rope=to(rope),
                         q_weight=to(wq), k_weight=to(wk), eps=eps, interleaved=pairs)
    torch.cuda.synchronize()
    at = pos.long().clamp(max=499)
    qr, qm = _ref_rows(q, wq, rope, at, eps, pairs)
    kr, km_ = _ref_rows(k, wk, rope, at, eps, pairs)
    assert bool((out[dead.to(DEV)] == 0).all())
    _near_rows(out.cpu()[~dead], qr[~dead], qm[~dead], dt, D)
    live = slots[~dead].long()
    kn, vn = kc.cpu().clone(), vc.cpu().clone()
    _near_rows(kn[live // p, live % p], kr[~dead], km_[~dead], dt, D)
    assert torch.equal(vn[live // p, live % p], v[~dead])
    kn[live // p, live % p], vn[live // p, live % p] = kc0[live // p, live % p], vc0[live // p, live % p]
    assert torch.equal(kn, kc0) and torch.equal(vn, vc0)  # nothing else was written


def test_append_in_place_keys_only_and_extremes():
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn(6, 4, 64, generator=g).to(BF), torch.randn(6, 2, 64, generator=g).to(BF)
    q[0] = 0                         # a row of zeros: eps alone
    q[1, 0] = 3e38                   # squares overflow fp32: mean is inf, the row becomes 0
    k[2, 1, 5] = float("inf")
    w = torch.ones(64)
    kc = torch.zeros(1, 16, 2, 64, dtype=BF, device=DEV)
    qd = q.to(DEV)
    out = kvcache.append(qd, k.to(DEV), None, kc, None, None, q_weight=w.to(DEV), k_weight=None, out=qd)
    assert out is qd
    qr, qm = _ref_rows(q, w, None, None, 1e-6, False)
    keep = torch.ones(6, 4, dtype=torch.bool)
    keep[1, 0] = False
    _near_rows(out.cpu()[keep], qr[keep], qm[keep], BF, 64)
    assert bool((out[1, 0] == 0).all())
    assert torch.equal(kc.cpu()[0, :6], k)  # no norm, no rotation: as they are, slot t for token t
    kvcache.append(None, k.to(DEV), None, kc, None, None)
    kvcache.append(qd[:0], k[:0].to(DEV), None, kc, None, None)  # no tokens
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------------------ attend ----

class Case:
    """Random cache and queries of requests with (slots in the cache, new tokens); unheld slots are NaN."""

    def __init__(self, lens, hq, hkv, D, dt, p=16, window=0, weighted=False, layout="slots", seed=0, sharp=1.0):
        g = torch.Generator().manual_seed(seed + 17 * len(lens) + D)
        self.lens, self.hq, self.hkv, self.D, self.dt, self.p, self.window = lens, hq, hkv, D, dt, p, window
        T = sum(n for _, n in lens)
        need = [-(-s // p) for s, _ in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(lens), max(need + [0]) + 1), -1, dtype=torch.int32)
        shape = (pages, p, hkv, D)
        self.k, self.v = torch.full(shape, math.nan, dtype=dt), torch.full(shape, math.nan, dtype=dt)
        self.lw = torch.full((pages, hkv, p), math.nan) if weighted else None
        at = 0
        for r, (s, _) in enumerate(lens):
            self.table[r, :need[r]] = order[at:at + need[r]].to(torch.int32)
            for j in range(0, s, p):
                page, m = order[at + j // p], min(p, s - j)
                self.k[page, :m] = torch.randn(m, hkv, D, generator=g).to(dt)
                self.v[page, :m] = torch.randn(m, hkv, D, generator=g).to(dt)
                if weighted:
                    w = torch.randint(1, 40, (hkv, m), generator=g).float().log()
                    w[torch.rand(hkv, m, generator=g) < 0.15] = -math.inf
                    self.lw[page, :, :m] = w
            at += need[r]
        self.q = (torch.randn(T, hq, D, generator=g) * sharp).to(dt)
        self.scale, self.layout = D ** -0.5, layout

    def set(self, r, j, k=None, v=None, lw=None):
        """Slot j of request r: its key, value and weight (all heads)."""
        page, off = int(self.table[r, j // self.p]), j % self.p
        if k is not None:
            self.k[page, off] = k
        if v is not None:
            self.v[page, off] = v
        if lw is not None:
            self.lw[page, :, off] = lw

    def device(self):
        k, v = self.k.to(DEV), self.v.to(DEV)
        q = self.q.to(DEV)
        if self.layout == "heads":
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif self.layout == "joint":  # keys and values side by side, queries inside wider rows
            kv = torch.stack([k, v], dim=2)
            k, v = kv[:, :, 0], kv[:, :, 1]
            wide = torch.zeros(q.shape[0], self.hq + 3, self.D + 8, dtype=self.dt, device=DEV)
            wide[:, 1:1 + self.hq, :self.D] = q
            q = wide[:, 1:1 + self.hq, :self.D]
        start = torch.tensor([0] + [n for _, n in self.lens]).cumsum(0).to(torch.int32)
        return dict(q=q, k_cache=k, v_cache=v, block_table=self.table.to(DEV), query_start=start.to(DEV),
                    seq_lens=torch.tensor([s for s, _ in self.lens], dtype=torch.int32, device=DEV),
                    scale=self.scale, window=self.window, log_weight=None if self.lw is None else self.lw.to(DEV),
                    max_new=max([n for _, n in self.lens] + [0]))

    def reference(self):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
        T, G = self.q.shape[0], self.hq // self.hkv
        out, tol = (torch.zeros(T, self.hq, self.D, dtype=torch.float64) for _ in range(2))
        ltol = torch.zeros(T, self.hq, dtype=torch.float64)
        lse = torch.full_like(ltol, -math.inf)
        t0, u = 0, U[self.dt]
        for r, (s, n) in enumerate(self.lens):
            j = torch.arange(s)
            page = self.table[r].long()[j // self.p]
            held = (page >= 0) & (page < self.k.shape[0])
            page = torch.where(held, page, 0)
            for h in range(self.hkv):
                k, v = self.k[page, j % self.p, h].double(), self.v[page, j % self.p, h].double()
                lw = torch.zeros(s, dtype=torch.float64)
                if self.lw is not None:
                    lw = self.lw[page, h, j % self.p].double()
                for i in range(n):
                    pos = s - n + i
                    see = held & (j <= pos) & (lw > -math.inf)
                    if self.window:
                        see &= j > pos - self.window
                    if not bool(see.any()):
                        continue
                    q = self.q[t0 + i, h * G:(h + 1) * G].double()
                    kk, vv, ww = k[see], v[see], lw[see]
                    sc = self.scale * (q @ kk.t()) + ww
                    es = (self.D + 16) * E * self.scale * (q.abs() @ kk.abs().t()).max(1).values
                    es = es + 4 * E * ww.abs().clamp(max=1e4).max() + 8 * E * sc.abs().clamp(max=1e4).max(1).values
                    l = torch.logsumexp(sc, 1)
                    pr = torch.softmax(sc, 1)
                    count = int(see.sum())
                    row = (2.1 * u + 4 * es + (count / 32 + 64) * E)[:, None]
                    o = slice(h * G, (h + 1) * G)
                    out[t0 + i, o], lse[t0 + i, o] = pr @ vv, l
                    small = count * 2.0 ** -25 * vv.abs().max() if self.dt == FP else 0
                    tol[t0 + i, o] = row * (pr @ vv.abs()) + small + 1e-30
                    ltol[t0 + i, o] = es + (count / 32 + 64) * E + 4 * E * l.abs()
            t0 += n
        return out, lse, tol, ltol

    def check(self, **kw):
        print(f"[attend] lens={self.lens[:6]} hq={self.hq} hkv={self.hkv} D={self.D} {self.dt} page={self.p} "
              f"window={self.window} weighted={self.lw is not None} {self.layout}", flush=True)
        out, lse = kvcache.attend(**dict(self.device(), **kw), lse=True)
        torch.cuda.synchronize()
        ro, rl, to, tl = self.reference()
        got, gl = out.double().cpu(), lse.double().cpu()
        assert bool(((got - ro).abs() <= to).all()), ((got - ro).abs() - to).max()
        empty = rl == -math.inf
        assert bool((gl[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
        d = (gl[~empty] - rl[~empty]).abs() - tl[~empty]
        assert bool((d <= 0).all()), d.max()
        return out, lse


DECODE = [(1, 1), (2, 1), (31, 1), (32, 1), (33, 1), (100, 1), (128, 1), (129, 1), (700, 1), (5, 0), (0, 0), (0, 1)]
CHUNKS = [(200, 70), (64, 64), (1, 1), (131, 67), (300, 1), (90, 0), (40, 50), (257, 129)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("hq,hkv,D,p,window,weighted,layout", [
    (8, 2, 128, 16, 0, False, "slots"), (4, 4, 64, 32, 0, False, "heads"), (7, 1, 80, 16, 50, False, "joint"),
    (16, 1, 256, 64, 0, True, "slots"), (14, 2, 128, 16, 33, True, "heads"), (32, 1, 64, 128, 0, False, "slots"),
    (40, 1, 128, 16, 0, True, "slots"), (3, 1, 16, 16, 1, False, "slots"), (10, 2, 208, 32, 0, False, "joint")])
def test_attend_decode(dt, hq, hkv, D, p, window, weighted, layout):
    Case(DECODE, hq, hkv, D, dt, p, window, weighted, layout).check()


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("hq,hkv,D,p,window,weighted,layout", [
    (4, 1, 128, 16, 0, False, "slots"), (3, 3, 64, 32, 0, False, "heads"), (7, 1, 80, 16, 50, False, "joint"),
    (2, 1, 256, 64, 0, True, "slots"), (6, 2, 128, 16, 33, True, "heads"), (5, 1, 64, 128, 100, False, "slots"),
    (20, 1, 128, 16, 0, False, "slots"), (1, 1, 16, 16, 1, False, "slots"), (2, 2, 208, 32, 0, True, "joint")])
def test_attend_chunks(dt, hq, hkv, D, p, window, weighted, layout):
    Case(CHUNKS, hq, hkv, D, dt, p, window, weighted, layout).check()


@pytest.mark.parametrize("seed", range(24))
def test_attend_random_shapes(seed):
    r = random.Random(seed)
    hkv, group = r.choice([1, 2, 3]), r.choice([1, 2, 3, 5, 8, 12, 17])
    most = r.choice([1, 1, 2, 6, 40, 150])
    lens = []
    for _ in range(r.choice([1, 2, 5, 9])):
        s = int(math.exp(r.uniform(0, math.log(900))))
        lens.append((s, min(r.randint(0, most), s + r.choice([0, 0, 2]))))
    if not any(n for _, n in lens):
        lens[0] = (lens[0][0], 1)
    Case(lens, hkv * group, hkv, 16 * r.randint(1, 16), r.choice([BF, FP]), r.choice([16, 32, 64, 256]),
         r.choice([0, 0, 1, 17, 100, 5000]), r.random() < 0.4, r.choice(["slots", "heads", "joint"]), seed,
         sharp=r.choice([0.3, 1.0, 4.0])).check()


@pytest.mark.parametrize("n,hq", [(2, 8), (5, 3), (4, 8), (8, 4), (33, 1)])
def test_attend_few_new_tokens(n, hq):
    """Several new tokens of each request: the narrow and the wide decode launch and the smallest chunks."""
    Case([(200, n), (n, n), (77, n), (n + 1, n)], hq, 1, 128, BF).check()


def test_attend_divided_keys():
    """Long contexts of few rows: many parts of one row, joined."""
    Case([(9000, 1), (333, 1)], 8, 1, 64, BF, p=64).check()
    Case([(5000, 100)], 2, 1, 128, FP, p=16).check()
    Case([(5000, 100), (4000, 1), (7, 7)], 2, 1, 128, BF, p=16, window=2000).check()


def test_attend_more_queries_than_slots():
    """The first queries stand before the cache's first slot and see nothing."""
    Case([(3, 5), (0, 4), (20, 70)], 4, 2, 64, BF).check()


def test_attend_sharp_and_flat_rows():
    for n in (1, 80):
        Case([(500, n)], 4, 1, 128, BF, sharp=30.0).check()
        c = Case([(500, n)], 4, 1, 128, BF, sharp=0.0)
        c.check()


@pytest.mark.parametrize("n", [1, 5, 90])
def test_attend_weights_remove_and_lowest(n):
    """-inf removes a slot whatever it holds; the type's lowest value alone is a plain mean."""
    low = torch.finfo(torch.float32).min
    c = Case([(150, n), (60, n if n < 60 else 60)], 4, 2, 64, BF, weighted=True)
    for j in range(150):
        c.set(0, j, lw=low)
    for j in (0, 7, 40, 59):
        c.set(1, j, k=math.inf, v=math.nan, lw=-math.inf)
    c.check()
    for j in range(60):
        c.set(1, j, lw=-math.inf)
    c.check()
    # lowest weights beside ordinary ones count nothing
    for j in range(0, 150, 2):
        c.set(0, j, lw=0.0)
    c.check()


@pytest.mark.parametrize("n,hq", [(4, 4), (3, 8), (90, 4)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 40])
def test_attend_unseen_values_do_not_reach_a_row(n, hq, bad, window):
    """A token's infinite or NaN key and value reach the rows that see it, and no other."""
    c = Case([(150, n), (100, n)], hq, 2, 64, BF, window=window)
    clean = Case([(150, n), (100, n)], hq, 2, 64, BF, window=window)
    at = 150 - n + n // 2  # a new token in the middle of the chunk
    c.set(0, at, v=bad)
    out = kvcache.attend(**c.device()).double().cpu()
    want, _, tol, _ = clean.reference()
    sees = [150 - n + i >= at and (not window or 150 - n + i - window < at) for i in range(n)] + [False] * n
    for t, s in enumerate(sees):
        if s:
            assert not bool(torch.isfinite(out[t]).any()), t
        else:
            assert bool(((out[t] - want[t]).abs() <= tol[t]).all()), t
    if not math.isfinite(bad):
        c.set(0, at, v=0.0)
        c.set(0, at, k=math.nan)
        out = kvcache.attend(**c.device()).double().cpu()
        clean.set(0, at, v=0.0)
        want, _, tol, _ = clean.reference()
        for t, s in enumerate(sees):
            if s:
                assert bool(torch.isnan(out[t]).all()), t
            else:
                assert bool(((out[t] - want[t]).abs() <= tol[t]).all()), t


@pytest.mark.parametrize("n,hq", [(4, 4), (3, 8), (90, 4)])
def test_attend_values_that_all_rows_see_beside_ones_that_some_do(n, hq):
    """An infinite value just before the new tokens, in a tile that not all rows see whole, reaches every row."""
    for back in (1, 2, 20):
        c = Case([(150, n), (100, n)], hq, 2, 64, BF)
        c.set(0, 150 - n - back, v=math.inf)
        out = kvcache.attend(**c.device())
        assert bool((out[:n] == math.inf).all()) and bool(torch.isfinite(out[n:]).all())


@pytest.mark.parametrize("n", [1, 60])
def test_attend_pages_outside_the_cache_are_not_seen(n):
    c = Case([(200, n), (90, n)], 4, 2, 128, BF, weighted=n == 60)
    c.table[0, 2], c.table[0, 5], c.table[1, 0] = -1, c.k.shape[0], 2 ** 30
    c.check()
    d = c.device()
    d["block_table"] = d["block_table"][:, :4].contiguous()  # a table narrower than the lengths
    got = kvcache.attend(**d)
    c.table[:, 4:] = -1
    want = kvcache.attend(**c.device())
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 60])
def test_attend_infinite_value_beside_a_page_outside_the_cache(n):
    """16 slots that are not held share a tile with an infinite value that every row sees."""
    c = Case([(200, n)], 4, 2, 64, BF)
    c.set(0, 50, v=math.inf)
    c.table[0, 2] = -1
    out = kvcache.attend(**c.device())
    assert bool((out == math.inf).all())


def test_attend_query_starts_that_do_not_ascend():
    """Overlapping requests (an error of the caller) stay inside every buffer, and later calls are right."""
    c = Case([(3000, 40), (2000, 40), (900, 40), (100, 40)], 8, 2, 128, BF)
    d = c.device()
    for starts in ([0, 160, 0, 160, 0], [-5, 1000, 7, -7, 160], [160, 0, 160, 0, 160]):
        kvcache.attend(**dict(d, query_start=torch.tensor(starts, dtype=torch.int32, device=DEV), max_new=160))
    torch.cuda.synchronize()
    c.check()


def test_attend_rows_outside_requests_and_host_bounds():
    c = Case([(50, 1), (70, 1)], 4, 2, 64, BF)
    d = c.device()
    q = torch.cat([d["q"], d["q"][:1]])
    out = torch.full_like(q, 7.0)
    lse = torch.full((3, 4), 7.0, device=DEV)
    kvcache.attend(**dict(d, q=q, max_new=1), out=out, lse=lse)
    assert bool((out[2] == 7).all()) and bool((lse[2] == 7).all())
    assert torch.equal(out[:2], kvcache.attend(**d))
    a = kvcache.attend(**dict(d, max_new=None))  # T as the bound
    assert torch.equal(a, out[:2])
    empty = kvcache.attend(**dict(d, q=d["q"][:0], query_start=torch.zeros_like(d["query_start"])))
    assert empty.shape[0] == 0


def test_attend_past_32_bit_offsets():
    """Pages whose elements lie beyond 2^32 from the start of the cache (keys and values in one 18 GB tensor)."""
    p, hkv, D = 64, 8, 128
    pages = (1 << 32) // (p * hkv * D) + 9
    big = torch.empty(pages, 2, p, hkv, D, dtype=BF, device=DEV)
    k, v = big[:, 0], big[:, 1]
    g = torch.Generator().manual_seed(5)
    use = [pages - 1, 3, pages - 5, pages // 2 + 1]
    kk, vv = torch.randn(4, p, hkv, D, generator=g).to(BF), torch.randn(4, p, hkv, D, generator=g).to(BF)
    for i, pg in enumerate(use):
        kvcache.append(None, kk[i].to(DEV), vv[i].to(DEV), k, v,
                       torch.arange(pg * p, pg * p + p, dtype=torch.int32, device=DEV))
    for n in (1, 40):
        c = Case([(4 * p - 7, n)], 16, hkv, D, BF, p=p)
        c.k, c.v = torch.cat([kk, kk[:2]]), torch.cat([vv, vv[:2]])
        c.table[0, :4] = torch.arange(4, dtype=torch.int32)
        d = dict(c.device(), k_cache=k, v_cache=v)
        d["block_table"][0, :4] = torch.tensor(use, dtype=torch.int32)
        out, lse = kvcache.attend(**d, lse=True)
        ro, rl, to, tl = c.reference()
        assert bool(((out.double().cpu() - ro).abs() <= to).all())
        assert bool(((lse.double().cpu() - rl).abs() <= tl).all())


@pytest.mark.parametrize("lens", [[(3000, 1), (200, 60), (900, 33)], DECODE, [(129, 1), (700, 1)], [(300, 2)]], ids=len)
def test_attend_same_bits_again_and_on_another_stream(lens):
    """With a workspace of any content, on a stream of its own."""
    c = Case(lens, 8, 2, 128, BF)
    a, la = c.check()
    ws = kvcache.Workspace(DEV)
    s = torch.cuda.Stream()
    d = c.device()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for fill in (0, 0xff, 0x7f, 0x3f):
            if ws.buf is not None:
                ws.buf.fill_(fill)
            b, lb = kvcache.attend(**d, lse=True, ws=ws)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_step_in_a_graph():
    """tables, append and attend captured once and replayed between eager work; each replay equals the eager step."""
    g = torch.Generator().manual_seed(9)
    p, hq, hkv, D, R = 16, 8, 2, 64, 3
    ctx, new = [40, 0, 133], [1, 20, 1]
    T = sum(new)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    k0 = torch.randn(40, p, hkv, D, generator=g).to(BF).to(DEV)
    v0 = torch.randn(40, p, hkv, D, generator=g).to(BF).to(DEV)
    table0 = torch.full((R, 12), -1, dtype=torch.int32, device=DEV)
    table0[0, :3], table0[2, :9] = i32([5, 1, 7]), i32(list(range(10, 19)))
    x = torch.randn(T, hq + 2 * hkv, D, generator=g).to(BF).to(DEV)
    rope, w = _rope(200, D).to(DEV), torch.ones(D, device=DEV)
    c, n, free = i32(ctx), i32(new), i32(list(range(20, 30)))
    ws = kvcache.Workspace(DEV)
    k, v, table = k0.clone(), v0.clone(), table0.clone()

    def step():
        t = kvcache.tables(c, n, table, free, p, T)
        q = kvcache.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], k, v, t.slots, positions=t.positions,
                           rope=rope, q_weight=w, k_weight=w)
        return kvcache.attend(q, k, v, table, t.query_start, t.seq_lens, lse=True, ws=ws) + (t.slots,)

    want = [t.clone() for t in step()]
    kw, vw, tw = k.clone(), v.clone(), table.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        k.copy_(k0), v.copy_(v0), table.copy_(table0)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + (k, v, table), want + [kw, vw, tw]):
            assert torch.equal(a, b)
        Case([(100, 3)], 4, 2, 64, FP).check()


# ---------------------------------------------------------------------------------------------------- refusals ----

def test_refusals():
    c = Case([(50, 1)], 4, 2, 64, BF)
    d = c.device()
    with pytest.raises(ValueError, match="shape"):
        kvcache.attend(**dict(d, q=d["q"][:, :, :32]))
    with pytest.raises(KMeansError, match="multiple of the cache's heads"):
        kvcache.attend(**dict(d, q=d["q"][:, :3].contiguous()))
    with pytest.raises(KMeansError, match="page_size"):
        kvcache.attend(**dict(d, k_cache=d["k_cache"][:, :8], v_cache=d["v_cache"][:, :8]))
    with pytest.raises(KMeansError, match="page_size"):
        kvcache.attend(**dict(d, k_cache=d["k_cache"].repeat(1, 3, 1, 1), v_cache=d["v_cache"].repeat(1, 3, 1, 1)))
    with pytest.raises(KMeansError, match="dim"):
        kvcache.attend(**dict(d, q=d["q"][..., :8].contiguous(), k_cache=d["k_cache"][..., :8].contiguous(),
                              v_cache=d["v_cache"][..., :8].contiguous()))
    with pytest.raises(KMeansError, match="16-byte aligned"):
        off = torch.zeros(d["q"].numel() + 1, dtype=BF, device=DEV)[1:].view_as(d["q"])
        kvcache.attend(**dict(d, q=off))
    with pytest.raises(KMeansError) as e:
        f = dict(d, q=d["q"].float(), k_cache=d["k_cache"].float(), v_cache=d["v_cache"].float())
        kvcache.attend(**f)
    assert e.value.status == 2
    with pytest.raises(KMeansError, match="window"):
        kvcache.attend(**dict(d, window=-1))
    with pytest.raises(KMeansError, match="scale"):
        kvcache.attend(**dict(d, scale=math.nan))
    with pytest.raises(ValueError, match="entries"):
        kvcache.attend(**dict(d, seq_lens=d["seq_lens"].repeat(2)))
    with pytest.raises(ValueError, match="int32"):
        kvcache.attend(**dict(d, query_start=d["query_start"].long()))
    with pytest.raises(ValueError, match="log_weight"):
        kvcache.attend(**dict(d, log_weight=torch.zeros(3, device=DEV)))
    k = d["k_cache"][:1, 0].contiguous()
    with pytest.raises(ValueError, match="together"):
        kvcache.append(None, k, None, d["k_cache"], None, None, rope=torch.zeros(4, 64, device=DEV))
    with pytest.raises(KMeansError, match="rot"):
        kvcache.append(None, k, None, d["k_cache"], None, None, rope=torch.zeros(4, 24, device=DEV),
                       positions=torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(KMeansError, match="eps"):
        kvcache.append(None, k, None, d["k_cache"], None, None, eps=-1.0)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(KMeansError, match="page_size"):
        kvcache.tables(i, i, d["block_table"], i, 24, 1)
    with pytest.raises(ValueError, match="total"):
        kvcache.tables(i, i, d["block_table"], i, 16, -1)

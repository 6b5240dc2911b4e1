// What the attention kernels share: how the work is divided, reductions
// across lanes, and the visibility of keys.  Internal to the library.
//
// Rows.  The queries of one request that read one cache head are n tokens x G
// query heads; row m of them is token m / G, head m % G.  A tile is BM rows.
//
// Division.  Lengths are on the device only, so every workgroup works out its
// share itself, from the lengths of all requests.
//   Decode launch: all keys of all requests and cache heads, in units of UNIT
//   keys, form one line, cut into as many equal pieces as there are
//   workgroups (as many as the GPU holds at once).  So all end together
//   whatever the lengths, and at most the first and the last request of a
//   piece are shared with another workgroup.
//   Chunk launch: a tile's keys are divided into ranges of `size` units, one
//   item per tile and range.  The size is the same for all requests: all the
//   launch's keys over `target` items, at least min_units.  A workgroup takes
//   the item of its own index; there are at most target + (number of tiles)
//   of them, a number that the host knows for its grid.
#pragma once

#include "kv_internal.hpp"

namespace kmkv {

constexpr int kWgThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// First key that the query at slot p and later ones see, rounded down to a
// whole unit.
template <int UNIT>
__device__ __forceinline__ int first_key(const AttendArgs& a, int p) {
  const int lo = a.window > 0 ? max(p - a.window + 1, 0) : 0;
  return lo - lo % UNIT;
}

struct Request {
  int q0, n;   // first query token, query tokens
  int seq, c;  // slots that its queries can see, slot of the first query (below 0 where there are more queries than
               // slots)
  int tiles;   // 0: not of this launch
  int units;   // key units of its longest tile, at least 1
};

template <int BM, int UNIT>
__device__ __forceinline__ Request request_of(const AttendArgs& a, int r) {
  Request q;
  const int end = a.query_start[r + 1];
  q.q0 = clampi(a.query_start[r], 0, a.T);
  q.n = clampi(end, q.q0, a.T) - q.q0;
  // (room is at most 2^30: positions and keys stay far from the ends of 32 bits)
  const int room = a.width << a.page_shift, sl = clampi(a.seq_lens[r], 0, 1 << 30);
  // (of more new tokens than T the first ones are here, and stand where they would with all)
  q.c = sl - min(max(end, q.q0) - q.q0, 1 << 30);
  q.seq = min(min(sl, q.c + q.n), room);
  const int64_t rows = (int64_t)q.n * a.G;
  q.tiles = rows > a.lo_rows && rows <= a.hi_rows ? (int)((rows + BM - 1) / BM) : 0;
  int64_t keys = q.seq;
  if (a.window > 0) {
    if (q.tiles == 1) {
      keys -= first_key<UNIT>(a, q.c);
    } else {
      const int64_t most = (int64_t)a.window + BM / a.G + 2 + UNIT;
      keys = keys < most ? keys : most;
    }
  }
  q.units = (int)((keys + UNIT - 1) / UNIT);
  q.units = max(q.units, 1);
  return q;
}

struct Item {
  Request q;
  int r, tile, split, splits, size;  // size: units of an item
  int part0;  // the request's first part: parts are the items of divided tiles, numbered alone (at most 2 * target,
              // since a divided tile of u units has at most 2 u / size of them)
  __device__ __forceinline__ int part() const { return part0 + tile * splits + split; }
};

// A piece of the decode launch's line of keys.  Positions count units; head h
// of a request that starts at unit u of a head's U is at h * U + u.
struct Line {
  int64_t per_head;    // U
  int64_t from, upto;  // this workgroup's piece
  int r, off, head;    // request and unit of it at `from`, head
  Request q;
};
// The line of `total` units in n <= total pieces: where piece i starts, and
// the piece that a position lies in.
__device__ __forceinline__ int64_t piece_start(int64_t i, int64_t total, int64_t n) { return i * total / n; }
__device__ __forceinline__ int64_t piece_of(int64_t pos, int64_t total, int64_t n) {
  return ((pos + 1) * n - 1) / total;
}

// The piece of workgroup i of n (of as many as there are units, where these
// are fewer); false where it has none.  Uniform over the workgroup of
// kWgThreads threads.  scratch: 32 8-byte words of LDS.
template <int BM, int UNIT>
__device__ __forceinline__ bool find_piece(const AttendArgs& a, int i, int n, Line& out, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.R + kWgThreads - 1) / kWgThreads;
  const int r0 = tid * per, r1 = min(r0 + per, a.R);
  Request q0 = {0, 0, 0, 0, 0, 0};
  if (r0 < r1) q0 = request_of<BM, UNIT>(a, r0);
  int64_t mine = q0.tiles ? q0.units : 0;
  for (int r = r0 + 1; r < r1; ++r) {
    const Request q = request_of<BM, UNIT>(a, r);
    mine += q.tiles ? q.units : 0;
  }
  double sum = wave_scan((double)mine);  // (exact below 2^53)
  if (lane == 63) scratch[wave] = (int64_t)sum;
  __syncthreads();
  int64_t last = (int64_t)sum, total = 0;
#pragma unroll
  for (int w = 0; w < kWgThreads / 64; ++w) {
    if (w < wave) last += scratch[w];
    total += scratch[w];
  }
  out.per_head = total;
  const int64_t all = total * a.Hkv, pieces = n < all ? n : all;
  if (i >= pieces) return false;
  out.from = piece_start(i, all, pieces);
  out.upto = piece_start(i + 1, all, pieces);
  out.head = (int)(out.from / total);
  const int64_t at = out.from - out.head * total;
  int64_t first = last - mine;
  if (at >= first && at < last) {  // this thread's requests hold the position
    for (int r = r0; r < r1; ++r) {
      const Request q = r == r0 ? q0 : request_of<BM, UNIT>(a, r);
      const int u = q.tiles ? q.units : 0;
      if (at < first + u) {
        const int v[8] = {r, (int)(at - first), q.q0, q.n, q.seq, q.c, q.tiles, q.units};
#pragma unroll
        for (int j = 0; j < 8; ++j) scratch[4 + j] = v[j];
        break;
      }
      first += u;
    }
  }
  __syncthreads();
  int v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_readfirstlane((int)scratch[4 + j]);
  out.r = v[0];
  out.off = v[1];
  out.q = Request{v[2], v[3], v[4], v[5], v[6], v[7]};
  return true;
}

// The next request of the launch after request r, the first again after the
// last (*head moves on).  There is one.  Uniform over the wavefront.
template <int BM, int UNIT>
__device__ __forceinline__ Request next_request(const AttendArgs& a, int& r, int& head) {
  const int lane = threadIdx.x & 63;
  int base = r + 1;
  for (;;) {
    if (base >= a.R) {
      base = 0;
      ++head;
    }
    Request q = {0, 0, 0, 0, 0, 0};
    if (base + lane < a.R) q = request_of<BM, UNIT>(a, base + lane);
    const uint64_t have = __ballot(q.tiles > 0);
    if (have) {
      const int l = __builtin_ctzll(have);
      r = base + l;
      return Request{__builtin_amdgcn_readlane(q.q0, l), __builtin_amdgcn_readlane(q.n, l),
                     __builtin_amdgcn_readlane(q.seq, l), __builtin_amdgcn_readlane(q.c, l),
                     __builtin_amdgcn_readlane(q.tiles, l), __builtin_amdgcn_readlane(q.units, l)};
    }
    base += 64;
  }
}

// The item of index `it`; false where there is none.  Uniform over the
// workgroup of kWgThreads threads.  scratch: 32 words of LDS.
template <int BM, int UNIT>
__device__ __forceinline__ bool find_item(const AttendArgs& a, int it, Item& out, int* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.R + kWgThreads - 1) / kWgThreads;
  const int r0 = tid * per, r1 = min(r0 + per, a.R);
  Request q0 = {0, 0, 0, 0, 0, 1};
  if (r0 < r1) q0 = request_of<BM, UNIT>(a, r0);
  // (fp32 sums: the size is rounded up by more than they can lose, so the bounds on items and parts hold)
  float cost = (float)q0.tiles * (float)q0.units;
  for (int r = r0 + 1; r < r1; ++r) {
    const Request q = request_of<BM, UNIT>(a, r);
    cost += (float)q.tiles * (float)q.units;
  }
  cost = wave_scan(cost);
  float* costs = (float*)scratch;
  if (lane == 63) costs[wave] = cost;
  if (tid == 0) scratch[16] = -1;
  __syncthreads();
  const float total = (costs[0] + costs[1]) + (costs[2] + costs[3]);
  const int size = max((int)fminf(total * 1.0001f / (float)a.target, 1e9f) + 1, a.min_units);
  // (A launch has fewer than 2^24 items; requests that overlap, an error of the caller, could have any number, so each
  // thread's count ends there and the sums stay below 2^32: an item belongs to one thread only.)
  constexpr unsigned kMost = (1u << 24) - 1;
  auto count = [&](const Request& q, unsigned& items, unsigned& parts) {
    const int splits = (q.units + size - 1) / size;
    const uint64_t n = (uint64_t)q.tiles * (unsigned)splits;
    items = n < kMost ? (unsigned)n : kMost;
    parts = splits > 1 ? items : 0u;
  };
  unsigned items, parts;
  count(q0, items, parts);
  for (int r = r0 + 1; r < r1; ++r) {
    unsigned i, p;
    count(request_of<BM, UNIT>(a, r), i, p);
    items = min(items + i, kMost);
    parts = min(parts + p, kMost);
  }
  unsigned last = wave_scan(items), plast = wave_scan(parts);
  if (lane == 63) {
    scratch[4 + wave] = (int)last;
    scratch[8 + wave] = (int)plast;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWgThreads / 64 - 1; ++w)
    if (w < wave) {
      last += (unsigned)scratch[4 + w];
      plast += (unsigned)scratch[8 + w];
    }
  unsigned first = last - items, pfirst = plast - parts;
  const unsigned at = (unsigned)it;
  if (at >= first && at < last) {  // this thread's requests hold the item
    for (int r = r0; r < r1; ++r) {
      const Request q = r == r0 ? q0 : request_of<BM, UNIT>(a, r);
      unsigned i, p;
      count(q, i, p);
      if (at - first < i) {
        const int v[9] = {r, (int)(at - first), (int)pfirst, q.q0, q.n, q.seq, q.c, q.tiles, q.units};
#pragma unroll
        for (int j = 0; j < 9; ++j) scratch[16 + j] = v[j];
        break;
      }
      first += i;
      pfirst += p;
    }
  }
  __syncthreads();
  int v[9];
#pragma unroll
  for (int j = 0; j < 9; ++j) v[j] = __builtin_amdgcn_readfirstlane(scratch[16 + j]);
  if (v[0] < 0) return false;
  out.r = v[0];
  out.part0 = v[2];
  out.q = Request{v[3], v[4], v[5], v[6], v[7], v[8]};
  out.size = size;
  out.splits = (out.q.units + size - 1) / size;
  const int k = v[1] / out.splits;
  out.tile = out.q.tiles - 1 - k;  // (last rows first: they see the most keys)
  out.split = v[1] - k * out.splits;
  return true;
}

// The keys of `size` units from unit `off` of those that rows of tokens
// i0 .. i1 see at all.
template <int UNIT>
__device__ __forceinline__ void key_range(const AttendArgs& a, const Request& q, int i0, int i1, int64_t off,
                                          int64_t size, int& k0, int& k1) {
  const int hi = max(min(q.seq, q.c + i1 + 1), 0);
  const int64_t s0 = first_key<UNIT>(a, q.c + i0) + off * UNIT, s1 = s0 + size * UNIT;
  k0 = (int)(s0 < hi ? s0 : hi);
  k1 = (int)(s1 < hi ? s1 : hi);
}

// A page and whether it is one of the cache's; page 0 stands for those that
// are not, so that loads from it stay in bounds.
__device__ __forceinline__ int page_of(const AttendArgs& a, const int32_t* row, int key, bool& ok) {
  const int col = key >> a.page_shift;
  const int p = (unsigned)col < (unsigned)a.width ? row[col] : -1;
  ok = p >= 0 && p < a.pages;
  return ok ? p : 0;
}
// The same for a key that is uniform over the wavefront: a scalar load (the
// kernels do not write the table), which does not wait for the vector loads
// in flight.
__device__ __forceinline__ int page_of_uniform(const AttendArgs& a, const int32_t* row, int key, bool& ok) {
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const int col = __builtin_amdgcn_readfirstlane(key) >> a.page_shift;
  const int p = (unsigned)col < (unsigned)a.width ? ((table_t)(uintptr_t)row)[col] : -1;
  ok = p >= 0 && p < a.pages;
  return ok ? p : 0;
}

// Largest and sum over the lanes l, l ^ 32 (and l ^ 16).
__device__ __forceinline__ float max32(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float max16(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float sum32(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float sum16(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// A product that is rounded by itself.  (Scores and their maximum: were one of
// them part of a fused difference, a maximum of 2^28 could be 16 below its own
// score, whose term 2^16 is more than fp16 holds.)
__device__ __forceinline__ float product(float x, float y) {
#pragma clang fp contract(off)
  return x * y;
}

// Scores are in units of log 2, so that 2^(s - m) takes no product; with
// weights they are natural, since log2(e) times a weight of the type's lowest
// value would overflow (a row of such keys is their plain mean, and its lse
// that value).  Factor of a score or of a maximum, against another:
template <bool NAT>
__device__ __forceinline__ float factor(float s, float m) {
  return exp2_(NAT ? (s - m) * kLog2e : s - m);
}
// The softmax term of a score, times 2^kTerm.
template <class T, bool NAT>
__device__ __forceinline__ float term(float s, float m) {
  if constexpr (T::kTerm == 0.f)
    return factor<NAT>(s, m);
  else
    return exp2_(NAT ? fmaf(s - m, kLog2e, T::kTerm) : (s - m) + T::kTerm);
}
// The natural logarithm of a sum l of terms relative to m.
template <class T, bool NAT>
__device__ __forceinline__ float log_sum(float m, float l) {
  const float e = __log2f(l * __builtin_ldexpf(1.f, -(int)T::kTerm));
  return NAT ? m + e * kLn2 : (m + e) * kLn2;
}

// Whether an element of the packed pair is infinite or NaN.
template <class T>
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & T::kExp) == T::kExp || ((w >> 16) & T::kExp) == T::kExp;
}
// The pair times 0: NaN for such elements.
template <class T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t w) {
  return ((w & T::kExp) == T::kExp ? 0x7fffu : 0u) | (((w >> 16) & T::kExp) == T::kExp ? 0x7fff0000u : 0u);
}
// The pair with such elements replaced by 0.
template <class T>
__device__ __forceinline__ uint32_t even_pair(uint32_t w) {
  if ((w & T::kExp) == T::kExp) w &= 0xffff0000u;
  if (((w >> 16) & T::kExp) == T::kExp) w &= 0xffffu;
  return w;
}

}  // namespace kmkv

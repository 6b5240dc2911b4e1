// What the attention kernels share: how the work is divided, reductions
// across lanes, and the visibility of keys.  Internal to the library.
//
// Rows.  The queries of one request that read one cache head are n tokens x G
// query heads; row m of them is token m / G, head m % G.  A tile is BM rows.
//
// Items.  A tile's keys are divided into ranges of `size` units, one item per
// tile and range.  The size is the same for all requests, so that items cost
// alike whatever the lengths: all the launch's keys over `target` items, at
// least min_units.  Lengths are on the device only, so every workgroup works
// out the division itself, from the lengths of all requests, and takes the
// item of its own index; there are at most target + (number of tiles) of
// them, a number that the host knows for its grid.
#pragma once

#include "kv_internal.hpp"

namespace kmkv {

constexpr int kWgThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

struct Request {
  int q0, n;   // first query token, query tokens
  int seq, c;  // slots in the cache, slot of the first query (below 0 where there are more queries than slots)
  int tiles;   // 0: not of this launch
  int units;   // key units of its longest tile, at least 1
};

template <int BM, int UNIT>
__device__ __forceinline__ Request request_of(const AttendArgs& a, int r) {
  Request q;
  q.q0 = clampi(a.query_start[r], 0, a.T);
  q.n = clampi(a.query_start[r + 1], q.q0, a.T) - q.q0;
  const int64_t room = (int64_t)a.width << a.page_shift;
  const int sl = max(a.seq_lens[r], 0);
  q.seq = (int64_t)sl > room ? (int)room : sl;
  q.c = sl - q.n;
  const int64_t rows = (int64_t)q.n * a.G;
  q.tiles = rows > a.lo_rows && rows <= a.hi_rows ? (int)((rows + BM - 1) / BM) : 0;
  int64_t keys = q.seq;
  if (a.window > 0) {
    const int64_t most = (int64_t)a.window + BM / a.G + 2 + UNIT;
    keys = keys < most ? keys : most;
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

// A request's items, and in the upper 32 bits those of them that are parts.
__device__ __forceinline__ int64_t items_of(const Request& q, int size) {
  const int splits = (q.units + size - 1) / size;
  const int64_t n = (int64_t)q.tiles * splits;
  return splits > 1 ? n | (n << 32) : n;
}

// The item of index `it`; false where there is none.  Uniform over the
// workgroup of kWgThreads threads.  scratch: 16 8-byte words of LDS.
template <int BM, int UNIT>
__device__ __forceinline__ bool find_item(const AttendArgs& a, int it, Item& out, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.R + kWgThreads - 1) / kWgThreads;
  const int r0 = tid * per, r1 = min(r0 + per, a.R);
  Request q0 = {0, 0, 0, 0, 0, 1};
  if (r0 < r1) q0 = request_of<BM, UNIT>(a, r0);
  int64_t cost = (int64_t)q0.tiles * q0.units;
  for (int r = r0 + 1; r < r1; ++r) {
    const Request q = request_of<BM, UNIT>(a, r);
    cost += (int64_t)q.tiles * q.units;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) cost += __shfl_xor(cost, d);
  if (lane == 0) scratch[wave] = cost;
  __syncthreads();
  const int64_t total = scratch[0] + scratch[1] + scratch[2] + scratch[3];
  const int64_t even = (total + a.target - 1) / a.target;
  const int size = (int)(even > a.min_units ? even : a.min_units);
  int64_t mine = items_of(q0, size);
  for (int r = r0 + 1; r < r1; ++r) mine += items_of(request_of<BM, UNIT>(a, r), size);
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  int64_t* waves = scratch + 4;
  int* found = (int*)(scratch + 8);
  if (lane == 63) waves[wave] = sum;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += waves[w];
  int64_t first = sum - mine;
  if (it >= (int)first && it < (int)sum) {  // this thread's requests hold the item
    for (int r = r0; r < r1; ++r) {
      const int64_t n = items_of(r == r0 ? q0 : request_of<BM, UNIT>(a, r), size);
      if (it < (int)(first + n)) {
        found[0] = r;
        found[1] = it - (int)first;
        found[2] = (int)(first >> 32);
        break;
      }
      first += n;
    }
  }
  __syncthreads();
  const int r = __builtin_amdgcn_readfirstlane(found[0]);
  if (r < 0) return false;
  out.r = r;
  out.part0 = __builtin_amdgcn_readfirstlane(found[2]);
  out.q = request_of<BM, UNIT>(a, r);
  out.size = size;
  out.splits = (out.q.units + size - 1) / size;
  const int k = __builtin_amdgcn_readfirstlane(found[1]);
  out.tile = k / out.splits;
  out.split = k - out.tile * out.splits;
  return true;
}

// The keys that a tile's rows see at all: [lo, hi), lo a multiple of UNIT; and
// the part of them that is the item's.
template <int BM, int UNIT>
__device__ __forceinline__ void key_range(const AttendArgs& a, const Item& w, int& k0, int& k1) {
  const int i0 = w.tile * BM / a.G, i1 = min((w.tile * BM + BM - 1) / a.G, w.q.n - 1);
  const int hi = min(w.q.seq, w.q.c + i1 + 1);
  int lo = a.window > 0 ? max(w.q.c + i0 - a.window + 1, 0) : 0;
  lo -= lo % UNIT;
  const int64_t s0 = lo + (int64_t)w.split * w.size * UNIT, s1 = s0 + (int64_t)w.size * UNIT;
  k0 = (int)(s0 < hi ? s0 : max(hi, 0));
  k1 = (int)(s1 < hi ? s1 : max(hi, 0));
}

// A page and whether it is one of the cache's; page 0 stands for those that
// are not, so that loads from it stay in bounds.
__device__ __forceinline__ int page_of(const AttendArgs& a, const int32_t* row, int key, bool& ok) {
  const int col = key >> a.page_shift;
  const int p = col < a.width ? row[col] : -1;
  ok = p >= 0 && p < a.pages;
  return ok ? p : 0;
}
// The same for a key that is uniform over the wavefront: a scalar load (the
// kernels do not write the table), which does not wait for the vector loads
// in flight.
__device__ __forceinline__ int page_of_uniform(const AttendArgs& a, const int32_t* row, int key, bool& ok) {
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const int col = __builtin_amdgcn_readfirstlane(key) >> a.page_shift;
  const int p = col < a.width ? ((table_t)(uintptr_t)row)[col] : -1;
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

// Scores are in units of log 2, so that 2^(s - m) takes no product; with
// weights they are natural, since log2(e) times a weight of the type's lowest
// value would overflow (a row of such keys is their plain mean, and its lse
// that value).  Factor of a score or of a maximum, against another:
template <bool NAT>
__device__ __forceinline__ float factor(float s, float m) {
  return exp2_(NAT ? (s - m) * kLog2e : s - m);
}
// The natural logarithm of l terms relative to m.
template <bool NAT>
__device__ __forceinline__ float log_sum(float m, float l) {
  return NAT ? m + __log2f(l) * kLn2 : (m + __log2f(l)) * kLn2;
}

// Whether an element of the packed pair is infinite or NaN.
template <class T>
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & T::kExp) == T::kExp || ((w >> 16) & T::kExp) == T::kExp;
}
// The pair with such elements replaced by 0.
template <class T>
__device__ __forceinline__ uint32_t even_pair(uint32_t w) {
  if ((w & T::kExp) == T::kExp) w &= 0xffff0000u;
  if (((w >> 16) & T::kExp) == T::kExp) w &= 0xffffu;
  return w;
}

}  // namespace kmkv

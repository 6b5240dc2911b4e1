// Page and slot tables of a serving step, from request lengths.
//
// With P slots a page, request r holds have = ceil(ctx / P) pages and needs
// need = ceil((ctx + new) / P).  query_start and page_start are the exclusive
// sums of new and of need - have; entry e of the free list goes to the request
// r with page_start[r] <= e < page_start[r+1], as its page have + e -
// page_start[r]; token t belongs to the request with query_start[r] <= t <
// query_start[r+1].
//
// All of it is latency: a launch (3 us), the sums, one binary search and two
// dependent loads a token.  Up to 4,096 requests every workgroup makes the sums
// itself in LDS, so that one launch does: 8 requests take 3.0 us, 250 with
// 18,108 new tokens 4.7, 4,095 with 138,650 new tokens 10.8 (25 with the sums in
// a launch of one workgroup before it, as above 4,096: 9,001 take 27 + 9).  LDS
// arrays of 512 or 4,096 requests.
#include "kv_internal.hpp"

namespace kmkv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int pages_of(int64_t n, int shift) { return (int)((n + (1ll << shift) - 1) >> shift); }

// LDS arrays have a word free after every 32, so that threads that walk
// neighbouring stretches of them meet few banks twice.
__host__ __device__ constexpr int padded(int i) { return i + (i >> 5); }

// start(r) <= x < start(r+1); x lies in [0, start(R)).
template <class F>
__device__ __forceinline__ int owner(F&& start, int R, int x) {
  int lo = 0, hi = R;  // start(lo) <= x, x < start(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The two sums of all R requests, CH at a time: the workgroup stages their
// new tokens and pages in LDS, each thread adds up its neighbours, the
// workgroup sums the threads, and each thread gives its requests' sums to
// put(request, query start, page start).  part: 8 ints of LDS; n, np: padded(CH) + 1.
template <int CH, class F>
__device__ __forceinline__ void scan_requests(const TablesArgs& a, int* part, int* n, int* np, F&& put) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base_q = 0, base_p = 0;
  for (int r0 = 0; r0 < a.R; r0 += CH) {
    const int m = min(CH, a.R - r0);
#pragma unroll 8
    for (int i = tid; i < m; i += kThreads) {
      const int c = max(a.ctx[r0 + i], 0), f = max(a.fresh[r0 + i], 0);
      n[padded(i)] = f;
      np[padded(i)] = pages_of((int64_t)c + f, a.page_shift) - pages_of(c, a.page_shift);
    }
    __syncthreads();
    const int per = (m + kThreads - 1) / kThreads, i0 = min(tid * per, m), i1 = min(i0 + per, m);
    int q = 0, p = 0;
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
      q += n[padded(i)];
      p += np[padded(i)];
    }
    int last_q = wave_scan(q), last_p = wave_scan(p);
    if (lane == 63) {
      part[wave] = last_q;
      part[4 + wave] = last_p;
    }
    __syncthreads();
    q = base_q + last_q - q;
    p = base_p + last_p - p;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) {
        q += part[w];
        p += part[4 + w];
      }
      base_q += part[w];
      base_p += part[4 + w];
    }
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
      const int f = n[padded(i)], g = np[padded(i)];
      put(r0 + i, q, p);
      q += f;
      p += g;
    }
    __syncthreads();
  }
  if (tid == 0) put(a.R, base_q, base_p);
}

// LDS_R > 0: every workgroup makes the sums itself in LDS (R <= LDS_R), so
// the whole call is one launch; otherwise they are in query_start and
// page_start already.
template <int LDS_R>
__global__ __launch_bounds__(kThreads) void tables_kernel(TablesArgs a) {
  __shared__ int part[8];
  __shared__ int s_q[LDS_R > 0 ? padded(LDS_R) + 1 : 1], s_p[LDS_R > 0 ? padded(LDS_R) + 1 : 1];
  if constexpr (LDS_R > 0) {
    scan_requests<LDS_R>(a, part, s_q, s_p, [&](int r, int q, int p) {
      s_q[padded(r)] = q;
      s_p[padded(r)] = p;
    });
    __syncthreads();
    for (int r = blockIdx.x * kThreads + threadIdx.x; r <= a.R; r += gridDim.x * kThreads) {
      a.query_start[r] = s_q[padded(r)];
      a.page_start[r] = s_p[padded(r)];
      if (r < a.R) a.seq_lens[r] = max(a.ctx[r], 0) + max(a.fresh[r], 0);
    }
  }
  auto qs = [&](int r) { return LDS_R > 0 ? s_q[padded(r)] : a.query_start[r]; };
  auto ps = [&](int r) { return LDS_R > 0 ? s_p[padded(r)] : a.page_start[r]; };
  const int total = qs(a.R), taken = ps(a.R);
  const int64_t step = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t e = first; e < taken; e += step) {
    const int r = owner(ps, a.R, (int)e);
    const int64_t col = pages_of(max(a.ctx[r], 0), a.page_shift) + (e - ps(r));
    if (col >= 0 && col < a.width) a.table[r * a.table_stride + col] = e < a.num_free ? a.free_pages[e] : -1;
  }
  for (int64_t t = first; t < a.T; t += step) {
    int pos = 0, slot = -1;
    if (t < total) {
      const int r = owner(qs, a.R, (int)t);
      const int c = max(a.ctx[r], 0);
      const int at = c + ((int)t - qs(r));
      const int col = at >> a.page_shift, have = pages_of(c, a.page_shift);
      int page = -1;
      if ((unsigned)col < (unsigned)a.width) {  // (lengths whose sums pass 2^31 stay inside the table too)
        if (col < have) {
          page = a.table[r * a.table_stride + col];
        } else {  // (not from the table: another workgroup writes that entry)
          const int64_t e = (int64_t)ps(r) + (col - have);
          if (e >= 0 && e < a.num_free) page = a.free_pages[e];
        }
      }
      pos = at + (a.offset ? a.offset[r] : 0);
      // (the slots of a page beyond the last whole one below 2^31 would wrap into another's)
      if (page >= 0 && page < (1 << (31 - a.page_shift)))
        slot = (page << a.page_shift) + (at & ((1 << a.page_shift) - 1));
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

__global__ __launch_bounds__(kThreads) void scan_kernel(TablesArgs a) {
  constexpr int CH = 4096;
  __shared__ int part[8], n[padded(CH) + 1], np[padded(CH) + 1];
  scan_requests<CH>(a, part, n, np, [&](int r, int q, int p) {
    a.query_start[r] = q;
    a.page_start[r] = p;
    if (r < a.R) a.seq_lens[r] = max(a.ctx[r], 0) + max(a.fresh[r], 0);
  });
}

}  // namespace

hipError_t launch_tables(const TablesArgs& a, hipStream_t stream) {
  const int64_t work = a.T > a.R ? a.T : a.R;
  int64_t grid = (work + kThreads - 1) / kThreads;
  if (grid > 512) grid = 512;
  if (grid < 1) grid = 1;
  if (a.R <= 512) {
    tables_kernel<512><<<dim3((unsigned)grid), kThreads, 0, stream>>>(a);
  } else if (a.R <= 4096) {
    tables_kernel<4096><<<dim3((unsigned)grid), kThreads, 0, stream>>>(a);
  } else {
    scan_kernel<<<1, kThreads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    tables_kernel<0><<<dim3((unsigned)grid), kThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace kmkv

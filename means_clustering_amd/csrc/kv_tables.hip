// Page and slot tables of a serving step, from request lengths.
//
// With P slots a page, request r holds have = ceil(ctx / P) pages and needs
// need = ceil((ctx + new) / P).  query_start and page_start are the exclusive
// sums of new and of need - have; entry e of the free list goes to the request
// r with page_start[r] <= e < page_start[r+1], as its page have + e -
// page_start[r]; token t belongs to the request with query_start[r] <= t <
// query_start[r+1].
#include "kv_internal.hpp"

namespace kmkv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int pages_of(int64_t n, int shift) { return (int)((n + (1ll << shift) - 1) >> shift); }

// Inclusive sum over the workgroup of two values per thread; `tot` gets the
// totals.  part: 2 * kThreads / 64 ints of LDS.
__device__ __forceinline__ void block_scan2(int& a, int& b, int& tot_a, int& tot_b, int* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int ua = __shfl_up(a, d), ub = __shfl_up(b, d);
    if (lane >= d) {
      a += ua;
      b += ub;
    }
  }
  if (lane == 63) {
    part[2 * wave] = a;
    part[2 * wave + 1] = b;
  }
  __syncthreads();
  tot_a = tot_b = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w == wave) {
      a += tot_a;
      b += tot_b;
    }
    tot_a += part[2 * w];
    tot_b += part[2 * w + 1];
  }
  __syncthreads();
}

// start[r] <= x < start[r+1]; x lies in [0, start[R]).
__device__ __forceinline__ int owner(const int* start, int R, int x) {
  int lo = 0, hi = R;  // start[lo] <= x, x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The two sums of all R requests, in chunks of kThreads requests.
template <class F>
__device__ __forceinline__ void scan_requests(const TablesArgs& a, int* part, F&& put) {
  int base_q = 0, base_p = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    int n = 0, np = 0, c = 0;
    if (r < a.R) {
      c = max(a.ctx[r], 0);
      n = max(a.fresh[r], 0);
      np = pages_of((int64_t)c + n, a.page_shift) - pages_of(c, a.page_shift);
    }
    int q = n, p = np, tq, tp;
    block_scan2(q, p, tq, tp, part);
    if (r < a.R) put(r, c, n, base_q + q - n, base_p + p - np);
    base_q += tq;
    base_p += tp;
  }
  if (threadIdx.x == 0) put(a.R, 0, 0, base_q, base_p);
}

// LDS_R > 0: every workgroup makes the sums itself in LDS (R <= LDS_R), so
// the whole call is one launch; otherwise they are in query_start and
// page_start already.
template <int LDS_R>
__global__ __launch_bounds__(kThreads) void tables_kernel(TablesArgs a) {
  __shared__ int part[2 * kThreads / 64];
  __shared__ int s_q[LDS_R > 0 ? LDS_R + 1 : 1], s_p[LDS_R > 0 ? LDS_R + 1 : 1];
  const int *qs = a.query_start, *ps = a.page_start;
  if constexpr (LDS_R > 0) {
    scan_requests(a, part, [&](int r, int c, int n, int q, int p) {
      s_q[r] = q;
      s_p[r] = p;
      if ((r / kThreads) % gridDim.x == blockIdx.x) {  // each workgroup writes its share
        a.query_start[r] = q;
        a.page_start[r] = p;
        if (r < a.R) a.seq_lens[r] = c + n;
      }
    });
    __syncthreads();
    qs = s_q;
    ps = s_p;
  }
  const int total = qs[a.R], taken = ps[a.R];
  const int64_t step = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t e = first; e < taken; e += step) {
    const int r = owner(ps, a.R, (int)e);
    const int64_t col = pages_of(max(a.ctx[r], 0), a.page_shift) + (e - ps[r]);
    if (col < a.width) a.table[r * a.table_stride + col] = e < a.num_free ? a.free_pages[e] : -1;
  }
  for (int64_t t = first; t < a.T; t += step) {
    int pos = 0, slot = -1;
    if (t < total) {
      const int r = owner(qs, a.R, (int)t);
      const int c = max(a.ctx[r], 0);
      const int at = c + ((int)t - qs[r]);
      const int col = at >> a.page_shift, have = pages_of(c, a.page_shift);
      int page = -1;
      if (col < a.width) {
        if (col < have) {
          page = a.table[r * a.table_stride + col];
        } else {  // (not from the table: another workgroup writes that entry)
          const int64_t e = (int64_t)ps[r] + (col - have);
          if (e < a.num_free) page = a.free_pages[e];
        }
      }
      pos = at + (a.offset ? a.offset[r] : 0);
      if (page >= 0) slot = (page << a.page_shift) + (at & ((1 << a.page_shift) - 1));
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

__global__ __launch_bounds__(kThreads) void scan_kernel(TablesArgs a) {
  __shared__ int part[2 * kThreads / 64];
  scan_requests(a, part, [&](int r, int c, int n, int q, int p) {
    a.query_start[r] = q;
    a.page_start[r] = p;
    if (r < a.R) a.seq_lens[r] = c + n;
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

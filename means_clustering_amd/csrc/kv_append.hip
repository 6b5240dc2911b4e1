// Norm, rotation and cache write of new queries, keys and values.
//
//   y = x / sqrt(mean(x^2) + eps) * weight,  (a, b) -> (a c - b s, b c + a s)
//
// A row is one head of one token.  Each lane holds two 16-byte chunks of it:
// for rotation in halves chunk u and its partner chunk u + rot/16, so a pair
// never crosses lanes, otherwise two neighbouring chunks.  The lanes of a row
// sum their squares by exchanges in the wavefront; everything else is private
// to the lane, and the row is read and written once.  Rows are read in fp32
// and rounded once.
//
// Memory bounds it: 16,384 tokens of 32 + 8 + 8 heads of 128 (403 MB, and a
// table row of 512 bytes a token that its heads share) take 75.8 us, 5.4 TB/s,
// where a large copy reaches 4.9; 5 tokens take 3.4 us, a launch and two
// dependent loads.  Rows of 80, 112 and 240 leave 3, 1 and 1 of 8, 8 and 16
// lanes idle and reach 3.9, 4.7 and 5.0 TB/s at such sizes.
#include "kv_internal.hpp"

namespace kmkv {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ void widen8(const u32x4_t& w, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = T::lo(w[i]);
    x[2 * i + 1] = T::hi(w[i]);
  }
}

template <class T>
__device__ __forceinline__ u32x4_t narrow8(const float* x) {
  return u32x4_t{T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7])};
}

// LPR: lanes per row, the power of two from D / 16 up.
template <class T, int LPR, bool PAIRS>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  constexpr int kRows = kThreads / LPR;
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LPR;
  const int u = threadIdx.x % LPR;
  if (row >= (int64_t)a.T * heads) return;  // (whole rows: the exchanges below stay inside a row)
  const int t = (int)(row / heads), h = (int)(row - (int64_t)t * heads);
  const int slot = a.slots ? a.slots[t] : t;
  const int pos = a.positions ? a.positions[t] : 0;
  const bool live = slot >= 0 && slot < a.num_slots && pos >= 0 && pos < a.max_pos;
  const int half = a.rot / 16;  // chunks of half the rotated part
  int c0, c1;                   // this lane's chunks
  bool turn;
  if (PAIRS) {
    c0 = 2 * u;
    c1 = c0 + 1;
    turn = c0 * 8 < a.rot;
  } else {
    turn = u < half;
    c0 = turn ? u : 2 * u;
    c1 = turn ? u + half : c0 + 1;
  }
  const bool mine = u * 16 < a.D;
  const int off = slot & ((1 << a.page_shift) - 1), page = slot >> a.page_shift;
  const uint16_t* src;
  uint16_t* dst;
  if (h < a.Hq) {
    src = a.q + t * a.q_token + h * a.q_head;
    dst = a.out + t * a.o_token + h * a.o_head;
    if (!live) {
      if (mine) {
        *(u32x4_t*)(dst + c0 * 8) = u32x4_t{0u, 0u, 0u, 0u};
        *(u32x4_t*)(dst + c1 * 8) = u32x4_t{0u, 0u, 0u, 0u};
      }
      return;
    }
  } else {
    if (!live) return;
    const int g = h - a.Hq;
    if (g < a.Hkv) {
      src = a.k + t * a.k_token + g * a.k_head;
      dst = a.kc + page * a.kc_page + off * a.kc_slot + g * a.kc_head;
    } else {
      if (!a.v) return;
      const int gv = g - a.Hkv;
      src = a.v + t * a.v_token + gv * a.v_head;
      dst = a.vc + page * a.vc_page + off * a.vc_slot + gv * a.vc_head;
      if (mine) {
        const u32x4_t w0 = *(const u32x4_t*)(src + c0 * 8), w1 = *(const u32x4_t*)(src + c1 * 8);
        *(u32x4_t*)(dst + c0 * 8) = w0;
        *(u32x4_t*)(dst + c1 * 8) = w1;
      }
      return;
    }
  }
  u32x4_t w0 = {0u, 0u, 0u, 0u}, w1 = w0;
  if (mine) {
    w0 = *(const u32x4_t*)(src + c0 * 8);
    w1 = *(const u32x4_t*)(src + c1 * 8);
  }
  float x[16];
  widen8<T>(w0, x);
  widen8<T>(w1, x + 8);
  const float* weight = h < a.Hq ? a.q_weight : a.k_weight;
  if (weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) ss += __shfl_xor(ss, d);
    const float inv = 1.0f / sqrtf(ss / (float)a.D + a.eps);
    if (mine) {
      const f32x4_t g0 = *(const f32x4_t*)(weight + c0 * 8), g1 = *(const f32x4_t*)(weight + c0 * 8 + 4);
      const f32x4_t g2 = *(const f32x4_t*)(weight + c1 * 8), g3 = *(const f32x4_t*)(weight + c1 * 8 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= inv * g0[i];
        x[4 + i] *= inv * g1[i];
        x[8 + i] *= inv * g2[i];
        x[12 + i] *= inv * g3[i];
      }
    }
  }
  if (turn && mine) {
    // 8 angles: those of chunk u's pairs (halves), or of the pairs in both chunks (interleaved)
    const float* cs = a.rope + (int64_t)pos * a.rot + u * 8;
    const float* sn = cs + a.rot / 2;
    const f32x4_t ca = *(const f32x4_t*)cs, cb = *(const f32x4_t*)(cs + 4);
    const f32x4_t sa = *(const f32x4_t*)sn, sb = *(const f32x4_t*)(sn + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = i < 4 ? ca[i & 3] : cb[i & 3], s = i < 4 ? sa[i & 3] : sb[i & 3];
      const int ia = PAIRS ? 2 * i : i, ib = PAIRS ? 2 * i + 1 : 8 + i;
      const float p = x[ia], r = x[ib];
      x[ia] = p * c - r * s;
      x[ib] = r * c + p * s;
    }
  }
  if (mine) {
    *(u32x4_t*)(dst + c0 * 8) = narrow8<T>(x);
    *(u32x4_t*)(dst + c1 * 8) = narrow8<T>(x + 8);
  }
}

template <class T, int LPR>
void launch_lpr(const AppendArgs& a, bool interleaved, hipStream_t stream) {
  const int64_t rows = (int64_t)a.T * (a.Hq + 2 * a.Hkv), per = kThreads / LPR;
  const dim3 grid((unsigned)((rows + per - 1) / per));
  if (interleaved)
    append_kernel<T, LPR, true><<<grid, kThreads, 0, stream>>>(a);
  else
    append_kernel<T, LPR, false><<<grid, kThreads, 0, stream>>>(a);
}

template <class T>
void launch_type(const AppendArgs& a, bool interleaved, hipStream_t stream) {
  if (a.D <= 32)
    launch_lpr<T, 2>(a, interleaved, stream);
  else if (a.D <= 64)
    launch_lpr<T, 4>(a, interleaved, stream);
  else if (a.D <= 128)
    launch_lpr<T, 8>(a, interleaved, stream);
  else
    launch_lpr<T, 16>(a, interleaved, stream);
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int dt, bool interleaved, hipStream_t stream) {
  if (dt == 1)
    launch_type<BF16>(a, interleaved, stream);
  else
    launch_type<F16>(a, interleaved, stream);
  return hipGetLastError();
}

}  // namespace kmkv

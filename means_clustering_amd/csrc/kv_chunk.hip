// Attention of many rows of each request over a paged cache: chunks of a
// prompt.  The same sums as the decode kernel,
//
//   s = scale * (K q) + weight,  m = running maximum, p = e^(s - m),
//   l = sum p,  o = sum p v,  out = o / l,
//
// bound by the matrix cores.  A workgroup takes 128 rows, 32 for each
// wavefront, and walks its keys in tiles of BN, staged through LDS for all
// four wavefronts: the next tile is copied straight to the other LDS buffer
// while this one is multiplied.  Two workgroups share a compute unit, so one's
// softmax runs beside the other's products.
//
// v_mfma_f32_32x32x16 with lane l = 32 h + x: the A operand's lane holds row
// x, depth 8 h .. 8 h + 7; B's column x, the same depths; the result's column
// x, rows 8 b + 4 h + i (b, i < 4).  As in the decode kernel S' = K Q' and
// O' = V' P', a lane's statistics belong to one query row, and P' is used as
// it comes out: depth 8 h + j of a 16-key step stands for key 8 (j / 4) + 4 h
// + j % 4.  V' comes in that order from the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns and each gets a
// column), so values are stored as they are in memory.
//
// LDS rows are DP elements; their 16-byte pieces are permuted by an exclusive
// or with a number that goes with the row, so that the lanes served in one
// cycle (256 bytes: 16 lanes' reads of K, one piece of 16 rows; 32 lanes'
// reads of V, 4 neighbouring pieces of 4 rows) meet no bank twice.
//
// Measured (MI355X, bf16, 32 + 8 heads of 128): 8,192 tokens over 32,768 slots
// 3.75-3.80 ms, 1,010-1,030 TFLOP/s, where torch's matrix products reach 1,190
// (8,192 square) to 1,362 (16,384 square); 509 tokens over 30,509 slots
// 273-317 us, 800-925 TFLOP/s.  The matrix cores are busy 49% of the time at 2.0 GHz, the
// vector units 47% (5.6 instructions for each of the 32 products of a tile and
// wavefront, one of them an exponential, at a quarter of the others' rate): in
// sum nearly all of it, so the two hardly overlap.
//   * Tiles copied to LDS directly, pages by scalar loads: 4.09 ms; through
//     registers 7.15 (they left none for reads ahead of the products).
//   * LDS pieces permuted for 256 bytes a cycle: no bank conflicts; by 8 rows
//     and pairs of pieces half of the LDS cycles were conflicts (1% slower).
//   * Reads of K 6 ahead of the products, the next 16 keys' terms made beside
//     a product of V: 3% together.
//   * Heaviest rows first: 1% here, 9% for 2 x 2,047 tokens of 32 + 32 heads.
//   * Scores a tile ahead, beside the softmax: 5% fewer cycles, but a lower
//     clock: 2% here, 4-11% slower for D = 64, D = 256 and with weights.
//   * D = 256 keeps one workgroup a compute unit and tiles of 32 keys (10%
//     faster than of 64): 4,096 tokens over 28,672 slots 4.70 ms, 760 TFLOP/s.
//   * Dims between 64, 128 and 256 multiply zeros in LDS: in the same case D =
//     80 668 TFLOP/s of its own products, 96 785, 192 588.
//   * fp16: terms times 2^14, 0.6% slower than without.
#include <type_traits>

#include "kv_attend.hpp"

namespace kmkv {
namespace {

constexpr int kLoadsDone = 0x0f70;  // s_waitcnt vmcnt(0)
// Kinds of instructions for the scheduler's groups.
constexpr int kSchedMfma = 0x008, kSchedLds = 0x100, kSchedValu = 0x402;
constexpr int kAhead = 6;  // reads of K ahead of the products

// Stands for the values of slots that no row sees: up to 256 elements.
__device__ const u32x4_t g_zeros[32] = {};

template <int CH>
__device__ __forceinline__ constexpr int k_turn(int row) {
  return CH == 8 ? (row >> 1) & 7 : row & 15;  // (of 8 pieces two rows lie side by side in the banks)
}
template <int CH>
__device__ __forceinline__ constexpr int v_turn(int row) {
  return CH == 8 ? (row & 2) * 2 : (row & 3) * 4;
}

template <class T>
__device__ __forceinline__ f32x16_t mfma32(const u32x4_t& a, const u32x4_t& b, const f32x16_t& c) {
  if constexpr (T::kExp == BF16::kExp)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

template <class T, int DP, bool LW>
__global__ __launch_bounds__(kWgThreads, DP == 256 ? 1 : 2) void chunk_kernel(AttendArgs a) {
  constexpr int BM = kChunkRows, BN = chunk_unit(DP);
  constexpr int KB = DP / 16;           // depth steps of K Q'
  constexpr int CH = DP / 8;            // 16-byte pieces of an LDS row
  constexpr int WR = BN / 4;            // rows of a tile that a wavefront copies
  constexpr int NI = WR * CH / 64;      // ... in this many instructions of 64 pieces
  constexpr int NT = BN / 32, DT = DP / 32;
  constexpr int TP = BN * CH;           // pieces of a tile
  __shared__ int scratch[32];
  __shared__ __align__(16) u32x4_t s_k[2 * TP];
  __shared__ __align__(16) u32x4_t s_v[2 * TP];
  __shared__ __align__(16) float s_w[3][LW ? BN : 4];  // weights, a tile ahead of the copies
  __shared__ int s_odd;  // a value was infinite or NaN in a tile that not all rows see, and taken out
  const int head = blockIdx.x % a.Hkv, it = blockIdx.x / a.Hkv;
  Item w;
  if (!find_item<BM, BN>(a, it, w, scratch)) return;
  if (w.splits > 1 && (unsigned)w.part() >= (unsigned)a.parts) return;  // (query_start is not ascending: no such part)
  const int tid = threadIdx.x, lane = tid & 63, x = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = w.q.n * a.G, c = w.q.c;
  const int tok0 = w.tile * BM / a.G, tok1 = min((w.tile * BM + BM - 1) / a.G, w.q.n - 1);
  if (head == 0 && w.split == 0)
    for (int i = tok0 + tid; i <= tok1; i += kWgThreads) a.info[w.q.q0 + i] = make_int4(w.part0, w.splits, i, 1);
  int k0, k1;
  key_range<BN>(a, w.q, tok0, tok1, (int64_t)w.split * w.size, w.size, k0, k1);
  const int32_t* row = a.table + w.r * a.table_stride;
  const int pmask = (1 << a.page_shift) - 1;

  // this lane's query row
  const int m = w.tile * BM + 32 * wave + x, mc = min(m, rows - 1);
  const int qi = mc / a.G, hq = head * a.G + (mc - qi * a.G);
  // (above 0, so that the largest product is the largest score; a scale of 0 makes zeros of the queries instead)
  const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
  u32x4_t qf[KB];
  {
    const uint16_t* qp = a.q + (int64_t)(w.q.q0 + qi) * a.q_token + hq * a.q_head + 8 * h;
    const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      qf[kb] = u32x4_t{0u, 0u, 0u, 0u};
      if (16 * kb + 8 * h < a.D) qf[kb] = *(const u32x4_t*)(qp + 16 * kb) ^ sign;
      if (a.scale == 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[kb][i] = zero_pair<T>(qf[kb][i]);
      }
    }
  }
  const int jmax = min(c + qi, k1 - 1), jmin = a.window > 0 ? c + qi - a.window + 1 : 0;
  // the wavefront's rows see keys of [see0, see1) at most, and all of [full0, full1); the workgroup's rows all
  // of [wfull0, wfull1)
  const int wq0 = __builtin_amdgcn_readfirstlane(min(w.tile * BM + 32 * wave, rows - 1) / a.G);
  const int wq1 = __builtin_amdgcn_readfirstlane(min(w.tile * BM + 32 * wave + 31, rows - 1) / a.G);
  const int full1 = min(c + wq0 + 1, k1), full0 = a.window > 0 ? c + wq1 - a.window + 1 : 0;
  const int see1 = min(c + wq1 + 1, k1), see0 = a.window > 0 ? c + wq0 - a.window + 1 : 0;
  const int wfull1 = min(c + tok0 + 1, k1), wfull0 = a.window > 0 ? c + tok1 - a.window + 1 : 0;

  f32x16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m_ = -INFINITY, l_ = 0.f;

  // Are all pages of the item's keys in the cache?  (Uniform.)
  bool hole = false;
  for (int j = (k0 >> a.page_shift) + tid; j <= (k1 - 1) >> a.page_shift; j += kWgThreads) {
    bool ok;
    (void)page_of(a, row, j << a.page_shift, ok);
    hole |= !ok;
  }
  const bool holes = __syncthreads_or(hole);
  if (a.D < DP) {  // pieces beyond the rows' end are not copied
    for (int i = tid; i < 2 * TP; i += kWgThreads) s_k[i] = s_v[i] = u32x4_t{0u, 0u, 0u, 0u};
  }
  if (tid == 0) s_odd = 0;
  __syncthreads();

  // Copies of a tile: the wavefront's rows lie in one page.
  auto page_at = [&](int kt) __attribute__((always_inline)) {
    bool ok;
    return page_of_uniform(a, row, kt + wave * WR, ok);
  };
  auto copy_rows = [&](int kt, int page, int buf, int wbuf, bool whole) __attribute__((always_inline)) {
    const int off = (kt + wave * WR) & pmask;
    const uint8_t* kp = a.k + page * a.k_page + head * a.k_head + off * a.k_slot;
    const uint8_t* vp = a.v + page * a.v_page + head * a.v_head + off * a.v_slot;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * (64 / CH) + lane / CH, pc = lane % CH;  // row of the wavefront's, piece of the LDS row
      const int at = buf * TP + (wave * NI + i) * 64;
      const int kr = wave * WR + r;
      const int kc = pc ^ k_turn<CH>(kr), vc = pc ^ v_turn<CH>(kr);
      if (whole || 8 * kc < a.D)
        __builtin_amdgcn_global_load_lds((const void*)(kp + (r * a.k_slot + kc * 16)),
                                         (__attribute__((address_space(3))) void*)(s_k + at), 16, 0, 0);
      const uint8_t* vr = vp + r * a.v_slot;
      if (LW && s_w[wbuf][kr] == -INFINITY) vr = (const uint8_t*)g_zeros;
      if (whole || 8 * vc < a.D)
        __builtin_amdgcn_global_load_lds((const void*)(vr + vc * 16),
                                         (__attribute__((address_space(3))) void*)(s_v + at), 16, 0, 0);
    }
  };
  auto copy = [&](int kt, int page, int buf, int wbuf) __attribute__((always_inline)) {
    if (a.D == DP)
      copy_rows(kt, page, buf, wbuf, true);
    else
      copy_rows(kt, page, buf, wbuf, false);
  };
  // Weights of a tile, one for each of the first BN threads.
  auto weight_at = [&](int kt) __attribute__((always_inline)) {
    bool ok;
    const int key = kt + tid, page = page_of(a, row, key, ok);
    const float v = a.lw[page * a.lw_page + head * a.lw_head + (key & pmask)];
    return ok && key < k1 ? v : -INFINITY;
  };
  // Takes out of the staged values what no row sees, whatever it is, and in a tile that not all rows see (`part`)
  // what is infinite or NaN.
  auto clean = [&](int kt, int buf, bool part) __attribute__((always_inline)) {
    bool odd = false;
    for (int i = tid; i < TP; i += kWgThreads) {
      const int r = i / CH, key = kt + r;
      bool in = key < k1;
      if (holes) {
        bool ok;
        (void)page_of(a, row, key, ok);
        in = in && ok;
      }
      if (!part && in) continue;
      u32x4_t v = s_v[buf * TP + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!in) v[j] = 0u;
        odd |= odd_pair<T>(v[j]);
        v[j] = even_pair<T>(v[j]);
      }
      s_v[buf * TP + i] = v;
    }
    if (odd) s_odd = 1;
  };

  // LDS addresses of this lane's operands: K's piece 2 kb + h of row x, V's 4 rows of 16 columns for each 32 columns
  int ka[KB], va[DT];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) ka[kb] = x * CH + ((2 * kb + h) ^ k_turn<CH>(x));
  {
    const int r = 4 * h + ((lane & 15) >> 2);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int col = 32 * d + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);  // elements
      va[d] = (r * CH + ((col >> 3) ^ v_turn<CH>(r))) * 16 + (col & 4) * 2;
    }
  }

  auto multiply = [&](int kt, int buf, int wbuf) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
    f32x16_t s[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) s[t] = mfma32<T>(s_k[buf * TP + 32 * t * CH + ka[kb]], qf[kb], s[t]);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedLds, kAhead, 0);
#pragma unroll
    for (int i = 0; i < NT * KB - kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedLds, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, kAhead, 0);
    __builtin_amdgcn_s_setprio(0);
    if (LW) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4_t wv = *(const f32x4_t*)&s_w[wbuf][32 * t + 8 * b + 4 * h];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = s[t][4 * b + i] * scale + wv[i];
            s[t][4 * b + i] = wv[i] == -INFINITY ? -INFINITY : v;  // (whatever the key is)
          }
        }
    }
    if (kt < full0 || kt + BN > full1 || holes) {
      uint32_t held = ~0u;  // bit g: keys 16 g .. 16 g + 15 of the tile lie in a page of the cache
      if (holes) {
#pragma unroll 1
        for (int g = 0; g < BN / 16; ++g) {
          bool ok;
          (void)page_of_uniform(a, row, kt + 16 * g, ok);
          if (!ok) held &= ~(1u << g);
        }
      }
      const int from = jmin - kt - 4 * h, upto = jmax - kt - 4 * h;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 32 * t + 8 * (i / 4) + (i & 3);
          const bool see = j >= from && j <= upto && ((held >> (2 * t + i / 8)) & 1);
          s[t][i] = see ? s[t][i] : -INFINITY;
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    mx = max32(mx);
    if (!LW) mx = product(mx, scale);
    const float mn = fmaxf(m_, mx), ms = mn == -INFINITY ? 0.f : mn;
    if (__any(mn > m_)) {
      const float al = factor<LW>(m_, ms);
      l_ *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= al;
      m_ = mn;
    }
    // the exponent of a term is score * factor + base; from 2^24 on the maximum's rounding shows in a fused sum:
    // product()
    float fac = scale, base = T::kTerm - ms;
    if (!LW && __any(fabsf(ms) >= 16777216.f)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = product(s[t][i], scale) - ms;
      fac = 1.f;
      base = T::kTerm;
    }
    float sum = 0.f;
    auto values = [&](int u, u32x4_t(&vf)[DT]) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const char* at = (const char*)s_v + va[d] + (buf * TP + (16 * u + 8 * e) * CH) * 16;
          const u32x2_t two = __builtin_bit_cast(
              u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)at));
          vf[d][2 * e] = two[0];
          vf[d][2 * e + 1] = two[1];
        }
    };
    auto terms = [&](int u, u32x4_t& pf) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = s[u / 2][8 * (u & 1) + j], e = LW ? term<T, LW>(v, ms) : exp2_(fmaf(v, fac, base));
        s[u / 2][8 * (u & 1) + j] = e;
        sum += e;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) pf[j] = T::pack(s[u / 2][8 * (u & 1) + 2 * j], s[u / 2][8 * (u & 1) + 2 * j + 1]);
    };
    // the values and terms of the next 16 keys are made while these are multiplied
    u32x4_t vf[2][DT], pf[2];
    values(0, vf[0]);
    terms(0, pf[0]);
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      if (u + 1 < 2 * NT) {
        values(u + 1, vf[(u + 1) & 1]);
        terms(u + 1, pf[(u + 1) & 1]);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mfma32<T>(vf[u & 1][d], pf[u & 1], o[d]);
      if (u + 1 < 2 * NT) {
        __builtin_amdgcn_sched_group_barrier(kSchedLds, 2 * DT, 0);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedValu, 32 / DT, 0);
        }
      }
    }
    l_ += sum;
  };

  int page = 0, wbuf = 0;
  if (k0 < k1) {
    if (LW) {
      if (tid < BN) {
        s_w[0][tid] = weight_at(k0);
        s_w[1][tid] = weight_at(k0 + BN);
      }
      __syncthreads();
    }
    copy(k0, page_at(k0), 0, 0);
    page = page_at(k0 + BN);
  }
  __builtin_amdgcn_s_waitcnt(kLoadsDone);
  __syncthreads();
  // One tile: the next is copied to the other buffer meanwhile.
  auto step = [&](int kt, auto b) __attribute__((always_inline)) {
    constexpr int buf = decltype(b)::value;
    const int wnext = wbuf == 2 ? 0 : wbuf + 1;
    const bool more = kt + BN < k1;
    float wn = 0.f;
    if (more) {
      copy(kt + BN, page, buf ^ 1, wnext);
      page = page_at(kt + 2 * BN);
      if (LW && tid < BN) wn = weight_at(kt + 2 * BN);
    }
    const bool part = kt < wfull0 || kt + BN > wfull1;
    if (part || holes) {
      clean(kt, buf, part);
      __syncthreads();
    }
    if (kt + BN > see0 && kt < see1) multiply(kt, buf, wbuf);
    if (LW && more && tid < BN) s_w[wnext == 2 ? 0 : wnext + 1][tid] = wn;
    wbuf = wnext;
    __builtin_amdgcn_s_waitcnt(kLoadsDone);
    __syncthreads();
  };
  for (int kt = k0; kt < k1; kt += 2 * BN) {
    step(kt, std::integral_constant<int, 0>{});
    if (kt + BN < k1) step(kt + BN, std::integral_constant<int, 1>{});
  }

  if (s_odd) {  // the values taken out, added to the rows that see them
#pragma unroll 1
    for (int key = k0; key < k1; ++key) {
      const int kt = key - key % BN;
      if (kt >= wfull0 && kt + BN <= wfull1) continue;  // (all rows see this tile: nothing was taken out)
      bool ok;
      const int page = page_of_uniform(a, row, key, ok), off = key & pmask;
      if (!ok || (LW && a.lw[page * a.lw_page + head * a.lw_head + off] == -INFINITY)) continue;
      const uint16_t* vp = (const uint16_t*)(a.v + page * a.v_page + off * a.v_slot + head * a.v_head);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = 32 * d + 8 * (i / 4) + 4 * h + (i & 3);
          const uint32_t v = e < a.D ? vp[e] : 0u;
          if ((v & T::kExp) == T::kExp && key >= jmin && key <= jmax) o[d][i] += T::lo(v);
        }
    }
  }

  const float L = sum32(l_);
  const float ms = m_ == -INFINITY ? 0.f : m_;
  if (m >= rows) return;
  if (w.splits == 1) {
    const int64_t tok = w.q.q0 + qi;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    uint16_t* op = a.out + tok * a.o_token + hq * a.o_head;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int e = 32 * d + 8 * b + 4 * h;
        if (e < a.D)
          *(u32x2_t*)(op + e) = u32x2_t{T::pack(o[d][4 * b] * inv, o[d][4 * b + 1] * inv),
                                        T::pack(o[d][4 * b + 2] * inv, o[d][4 * b + 3] * inv)};
      }
    if (a.lse && h == 0) a.lse[tok * a.Hq + hq] = log_sum<T, LW>(ms, L);
  } else {
    const int64_t at = ((int64_t)w.part() * a.Hkv + head) * BM + 32 * wave + x;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *(f32x4_t*)(a.part_o + at * DP + 32 * d + 8 * b + 4 * h) =
            f32x4_t{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
    if (h == 0) a.part_ml[at] = f32x2_t{m_, L};
  }
}

template <class T, int DP>
void chunk_lw(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.max_items * a.Hkv));
  if (a.lw)
    chunk_kernel<T, DP, true><<<grid, kWgThreads, 0, stream>>>(a);
  else
    chunk_kernel<T, DP, false><<<grid, kWgThreads, 0, stream>>>(a);
}

template <class T>
void chunk_dim(const AttendArgs& a, hipStream_t stream) {
  const int dp = dim_pad(a.D);
  if (dp == 64)
    chunk_lw<T, 64>(a, stream);
  else if (dp == 128)
    chunk_lw<T, 128>(a, stream);
  else
    chunk_lw<T, 256>(a, stream);
}

}  // namespace

hipError_t launch_chunk(const AttendArgs& a, int dt, hipStream_t stream) {
  if (dt == 1)
    chunk_dim<BF16>(a, stream);
  else
    chunk_dim<F16>(a, stream);
  return hipGetLastError();
}

}  // namespace kmkv

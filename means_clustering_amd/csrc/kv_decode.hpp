// Attention of few rows (at most 16 or 32 for each request and cache head)
// over a paged cache: the decode step.  (kv_join.hpp joins divided rows.)
//
//   s = scale * (K q) + weight,  m = running maximum, p = e^(s - m),
//   l = sum p,  o = sum p v,  out = o / l
//
// The cache is read once and that is what bounds it.  A wavefront takes 32
// keys at a time, its keys and values straight from memory into registers
// (one step ahead of the products), and keeps its own m, l and o; the four
// wavefronts of a workgroup take turns in the keys and are joined at the end.
//
// v_mfma_f32_16x16x32 with lane l = 16 g + x: the A operand's lane holds row
// x, depth 8 g .. 8 g + 7; B's holds column x, the same depths; the result's
// holds column x, rows 4 g .. 4 g + 3.  The first product is S' = K Q' (rows
// are keys, columns the query rows), the second O' = V' P', so a lane's
// maxima, sums and factors belong to one query row.  P' needs no exchange:
// the lane's results of two 16-key halves are the 8 depths of its group once
// depth 8 g + j stands for key 4 g + j of half 0 (j < 4) or key 4 g + j - 4
// of half 1.  V' has to follow that order: the lane loads DV neighbouring
// columns of those 8 keys, and a byte permute of two keys' words makes the
// operands of the columns' 16 lanes.
//
// What bounds it, measured (MI355X; a plain read of 1 GB reaches 6.3 TB/s, a
// copy 4.9): 64 requests of up to 8,191 slots with 8 heads of 128 read 847 MB
// in 155 us (5.5 TB/s), two of 131,000 slots with weights 428 MB in 83 us
// (5.1 TB/s), the join after them 5-6 us; a single request of 500 slots takes
// 8 us, the latencies of its lengths, pages and keys, and the join 3-4 more.
// 63 requests of 32 + 8 heads of 256 read 1.3 GB in 217 us (6.0 TB/s) without
// registers for a step ahead; of 80 (as 128, padding not read) 404 MB in 98.
//   * Equal pieces of one line of keys against items of equal size per
//     request: 255 requests of D = 64 149 us against 180, 63 requests of 5 new
//     tokens 176 against 195 (items leave the last round of workgroups short).
//   * Page numbers by scalar loads, a step ahead: 64 requests 175 us against
//     199 with vector loads, whose wait also waited for keys in flight.
//   * Values are read past the caches (non-temporal loads; a load's lanes take
//     whole lines, which nobody wants again): 64 requests 161 us against 176.
//     Keys are not: a load takes half of each line, so the other half is
//     wanted at once (both so: 164 us, a third more reads of the L2).
// P is rounded to the cache's type for the matrix cores: its relative error of
// 2^-8 (2^-11) is that of the result's own rounding.  In fp16 the terms are
// held times 2^14, or those below 2^-14 of the largest would lose bits and
// those below 2^-25 everything, though a long context can have most of its sum
// in them; so 2^-28 and 2^-39 are the limits.  m, l and o are fp32.
//
// An 8-bit cache is half the bytes: 64 requests of up to 8,191 slots with 8
// heads of 128 (424 MB) 84 us where 16 bits take 155.  gfx950 converts two codes
// and multiplies them by their block's scale in one instruction (vector units
// 35% busy), so what is left is a piece's fixed part, 7 us of lengths, pages,
// first keys and join.  Twice to four times as many pieces were slower.
//   * Loads of forms in no branch: behind one every wait is for all loads.
//   * A load of 16 codes is the operand of two products, with the queries'
//     depths in that order; of values, codes of two keys are paired by byte
//     permutes before they are widened, half as many as after it.
// Other scores over 16 bits, 63 requests (123 us without): a cap 129, slopes
// 134, a prefix 133; 31 requests of heads of 256 with a cap 111 (5.6 TB/s).
#pragma once

#include "kv_attend.hpp"

namespace kmkv {
namespace {

template <class T>
__device__ __forceinline__ f32x4_t mfma16(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
  if constexpr (T::kExp == BF16::kExp)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// One step's keys and values of a wavefront: 32 keys.  F8: codes of an 8-bit
// cache, four in a word, and the bytes of the halves' scales.
template <int DP, bool LW, bool F8 = false>
struct Tile {
  u32x4_t k[2][DP / (F8 ? 64 : 32)];
  uint32_t v[8][DP / (F8 ? 64 : 32)];  // 8 keys x DP / 16 columns
  f32x4_t w[LW ? 2 : 1];
  uint32_t ks[F8 ? 2 : 1], vs[F8 ? 2 : 1];
  bool ok[2];                          // (uniform) the halves' pages are in the cache
};

// Pages of a step's two halves (uniform): looked up a step before the loads
// that need them.
struct Pages {
  int page[2];
  bool ok[2];
};
__device__ __forceinline__ Pages pages_of(const AttendArgs& a, const int32_t* row, int k) {
  Pages p;
  p.page[0] = page_of_uniform(a, row, k, p.ok[0]);
  p.page[1] = page_of_uniform(a, row, k + 16, p.ok[1]);
  return p;
}

// WHOLE: rows are DP elements; otherwise the columns from a.D on count as 0.
// F8: an 8-bit cache.  A lane's load of 16 codes of a key is the operand of
// two products, the depths of whose queries follow it.
template <class T, int DP, int NQ, bool LW, bool WHOLE, bool F8 = false>
struct Decode {
  static constexpr int BM = 16 * NQ, KB = DP / 32, DV = DP / 16, VW = DP / 32;
  static constexpr int LS = DP + 4;  // LDS row of a wavefront's partial result, in floats
  // Neighbouring columns of a lane: one load, whose 16 lanes read whole rows of up to 128 columns.
  static constexpr int kRun = F8 || DV < 8 ? DV : 8;
  // The e-th column that lane x of a group loads.
  static __device__ __forceinline__ constexpr int column(int x, int e) {
    return e / kRun * (16 * kRun) + x * kRun + e % kRun;
  }

  // The first of the 8 depths of lane group g in product kb.
  static __device__ __forceinline__ constexpr int depth(int kb, int g) {
    return F8 ? kb / 2 * 64 + g * 16 + kb % 2 * 8 : kb * 32 + g * 8;
  }

  // The loads of forms have no branch: behind one whose loads may or may not
  // be in flight, every wait is for all of them.  Columns from a.D on are read
  // as the row's first (keys of these become zeros where they are used).  With
  // a lane below 0 all lanes read one place of a row, and nobody uses it.
  static __device__ __forceinline__ void load(const FormArgs& a, const Pages& pg, int head, int k, int lane,
                                              Tile<DP, LW, true>& t) {
    const int x = lane < 0 ? 0 : lane & 15, g = lane < 0 ? 0 : lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k + 16 * h;
      t.ok[h] = pg.ok[h];
      const int64_t page = pg.page[h];
      const int off = key & ((1 << a.page_shift) - 1);
      t.ks[h] = a.ks[page * a.ks_page + head * a.ks_head + (off >> 4)];
      t.vs[h] = a.vs[page * a.vs_page + head * a.vs_head + (off >> 4)];
      const uint8_t* kp = a.k + page * a.k_page + off * a.k_slot + head * a.k_head + (x * a.k_slot + g * 16);
#pragma unroll
      for (int c = 0; c < DP / 64; ++c)
        t.k[h][c] = *(const u32x4_t*)(kp + (WHOLE || c * 64 + g * 16 < a.D ? c * 64 : -g * 16));
      if (LW) t.w[h] = *(const f32x4_t*)(a.lw + page * a.lw_page + head * a.lw_head + off + 4 * g);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k + 16 * h;
      const int64_t page = pg.page[h];
      const int off = key & ((1 << a.page_shift) - 1);
      const uint8_t* vp = a.v + page * a.v_page + off * a.v_slot + head * a.v_head +
                          (4 * g * a.v_slot + (WHOLE || column(x, 0) < a.D ? x * kRun : 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t* d = t.v[4 * h + j];
        const uint8_t* s = vp + j * a.v_slot;
        if constexpr (DP == 64) {
          d[0] = __builtin_nontemporal_load((const uint32_t*)s);
        } else if constexpr (DP == 128) {
          const u32x2_t w = __builtin_nontemporal_load((const u32x2_t*)s);
          d[0] = w[0];
          d[1] = w[1];
        } else {
          const u32x4_t w = __builtin_nontemporal_load((const u32x4_t*)s);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = w[i];
        }
      }
    }
  }

  template <class A>
  static __device__ __forceinline__ void load(const A& a, const Pages& pg, int head, int k, int lane,
                                              Tile<DP, LW>& t) {
    const int x = A::kForm && lane < 0 ? 0 : lane & 15, g = A::kForm && lane < 0 ? 0 : lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k + 16 * h;
      t.ok[h] = pg.ok[h];
      const int64_t page = pg.page[h];
      const int off = key & ((1 << a.page_shift) - 1);
      const uint8_t* kp = a.k + page * a.k_page + off * a.k_slot + head * a.k_head + (x * a.k_slot + g * 16);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (A::kForm)
          t.k[h][kb] = *(const u32x4_t*)(kp + (WHOLE || kb * 32 + g * 8 < a.D ? kb * 64 : -g * 16));
        else if (WHOLE || kb * 32 + g * 8 < a.D)
          t.k[h][kb] = *(const u32x4_t*)(kp + kb * 64);
        else
          t.k[h][kb] = u32x4_t{0u, 0u, 0u, 0u};
      }
      if (LW) t.w[h] = *(const f32x4_t*)(a.lw + page * a.lw_page + head * a.lw_head + off + 4 * g);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k + 16 * h;
      const int64_t page = pg.page[h];
      const int off = key & ((1 << a.page_shift) - 1);
      const uint8_t* vp = a.v + page * a.v_page + off * a.v_slot + head * a.v_head +
                          (4 * g * a.v_slot + x * (kRun * 2));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t* d = t.v[4 * h + j];
        const uint8_t* s = vp + j * a.v_slot;
        if constexpr (DP == 64) {
          u32x2_t w = {0u, 0u};
          if (A::kForm)
            w = __builtin_nontemporal_load((const u32x2_t*)(s - (WHOLE || column(x, 0) < a.D ? 0 : x * (kRun * 2))));
          else if (WHOLE || column(x, 0) < a.D)
            w = __builtin_nontemporal_load((const u32x2_t*)s);
          d[0] = w[0];
          d[1] = w[1];
        } else {
#pragma unroll
          for (int c = 0; c < VW; c += 4) {
            u32x4_t w = {0u, 0u, 0u, 0u};
            if (A::kForm)
              w = __builtin_nontemporal_load((const u32x4_t*)(s + (WHOLE || column(x, 2 * c) < a.D
                                                                       ? column(0, 2 * c) * 2
                                                                       : -x * (kRun * 2))));
            else if (WHOLE || column(x, 2 * c) < a.D)
              w = __builtin_nontemporal_load((const u32x4_t*)(s + column(0, 2 * c) * 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) d[c + i] = w[i];
          }
        }
      }
    }
  }
};

// (A form, whose A is FormArgs, may have a cap, slopes and a prefix.)
template <class T, int DP, int NQ, bool LW, bool WHOLE, class A = AttendArgs, bool F8 = false>
__global__ __launch_bounds__(kWgThreads, decode_per_cu(DP, 16 * NQ)) void decode_kernel(A a) {
  using W = Decode<T, DP, NQ, LW, WHOLE, F8>;
  constexpr int BM = W::BM, KB = W::KB, DV = W::DV, LS = W::LS;
  constexpr int STAGES = decode_stages(DP, 16 * NQ, F8);
  __shared__ int64_t scratch[32];
  __shared__ float s_ml[4][BM][2];
  __shared__ __align__(16) float s_o[4][BM][LS];
  Line line;
  const bool some = find_piece<BM, kDecodeUnit>(a, blockIdx.x, gridDim.x, line, scratch);
  const int tid = threadIdx.x, lane = tid & 63, x = lane & 15, g = lane >> 4;
  if (blockIdx.x == 0 && tid == 0) *a.per_head = line.per_head;
  if (!some) return;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  struct {
    Request q;
    int r, head, off;
  } w = {line.q, line.r, line.head, line.off};
  int64_t pos = line.from;
  for (;;) {
    const int64_t left = line.upto - pos;
    const int len = w.q.units - w.off < left ? w.q.units - w.off : (int)left;
    const bool whole = len == w.q.units;
    const int part = 2 * (int)blockIdx.x + (pos == line.from ? 0 : 1);
    const int rows = w.q.n * a.G, c = w.q.c, head = w.head;
    if (head == 0 && w.off == 0)
      for (int i = tid; i < w.q.n; i += kWgThreads)
        a.info[w.q.q0 + i] = make_int4((int)(uint32_t)pos, w.q.units, i, (int)(pos >> 32) << 1);
    // numbers k0 .. k1 - 1 of keys, slots below `end`
    int k0, k1, end;
    Keys range;
    if constexpr (A::kForm) {
      range = form_range<kDecodeUnit>(a, w.q, w.r, 0, w.q.n - 1, w.off, len);
      k0 = range.k0;
      k1 = range.k1;
      end = range.end;
    } else {
      key_range<kDecodeUnit>(a, w.q, 0, w.q.n - 1, w.off, len, k0, k1);
      end = k1;
    }
    auto slot_of = [&](int k) __attribute__((always_inline)) {
      if constexpr (A::kForm)
        return range.slot(k);
      else
        return k;
    };
    const int32_t* row = a.table + w.r * a.table_stride;

    // queries: this lane's column of each group of 16 rows
    u32x4_t qf[NQ][KB];
    int jmin[NQ], jmax[NQ];
    float slope[A::kForm ? NQ : 1];
    int c_of[A::kForm ? NQ : 1];  // the query's slot
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int m = min(16 * q + x, rows - 1);
      const int i = m / a.G, hq = head * a.G + (m - i * a.G);
      const uint16_t* qp = a.q + (int64_t)(w.q.q0 + i) * a.q_token + hq * a.q_head + g * 8;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        qf[q][kb] = u32x4_t{0u, 0u, 0u, 0u};
        if constexpr (F8) {
          if (W::depth(kb, g) < a.D) qf[q][kb] = *(const u32x4_t*)(qp + (W::depth(kb, g) - g * 8));
        } else {
          if (kb * 32 + g * 8 < a.D) qf[q][kb] = *(const u32x4_t*)(qp + kb * 32);
        }
      }
      if constexpr (A::kForm) {
        slope[q] = a.slopes ? slope_of<LW>(a.slopes[hq]) : 0.f;
        c_of[q] = c + i;
      }
      jmax[q] = min(c + i, end - 1);
      jmin[q] = a.window > 0 ? c + i - a.window + 1 : 0;
    }
    // a step whose keys all rows see: from `full0`, up to `full1`
    const int full1 = min(c + 1, end), full0 = a.window > 0 ? c + w.q.n - a.window : 0;

    f32x4_t o[NQ][DV];
    float m_[NQ], l_[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m_[q] = -INFINITY;
      l_[q] = 0.f;
#pragma unroll
      for (int e = 0; e < DV; ++e) o[q][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    auto all_see = [&](int k) __attribute__((always_inline)) {
      if constexpr (A::kForm)
        return (k >= full0 && k + 32 <= full1) || k + 32 <= range.pre;
      else
        return k >= full0 && k + 32 <= full1;
    };
    auto sees = [&](int q, int key) __attribute__((always_inline)) {
      if constexpr (A::kForm)
        return (key >= jmin[q] && key <= jmax[q]) || key < range.pre;
      else
        return key >= jmin[q] && key <= jmax[q];
    };

    bool some_odd = false;
    // Takes out of a step's values what no row sees, whatever it is, and where rows differ in what they see what is
    // infinite or NaN: that is added in the end to the rows that see it.
    auto clean = [&](uint32_t(&v)[8][W::VW], const Tile<DP, LW, F8>& t, int k,
                     bool all) __attribute__((always_inline)) {
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = k + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
        bool in = (j < 4 ? t.ok[0] : t.ok[1]) && key < end;
        if (LW) in = in && t.w[j >> 2][j & 3] != -INFINITY;
#pragma unroll
        for (int i = 0; i < W::VW; ++i) {
          if (!in) v[j][i] = 0u;
          if (!all) odd |= odd_pair<T>(v[j][i]);
        }
      }
      if (__any(odd)) {
        some_odd = true;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < W::VW; ++i) v[j][i] = even_pair<T>(v[j][i]);
      }
    };
    auto process = [&](Tile<DP, LW, F8>& t, int k) __attribute__((always_inline)) {
      const bool all = all_see(k) && t.ok[0] && t.ok[1];
      if constexpr (!F8) {
        if (!all || LW) clean(t.v, t, k, all);
      }
      // (made here and not beside the loads, which they would wait for there)
      float fk[2], fv[2];
      if constexpr (F8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          asm volatile("" : "+v"(t.ks[h]), "+v"(t.vs[h]));
          fk[h] = block_scale(t.ks[h]);
          fv[h] = block_scale(t.vs[h]);
        }
      }
      u32x4_t pf[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float s[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            u32x4_t kf;
            if constexpr (F8) {
              const uint32_t w0 = t.k[h][kb / 2][kb % 2 * 2], w1 = t.k[h][kb / 2][kb % 2 * 2 + 1];
              kf = u32x4_t{code_pair<T, false>(w0, fk[h]), code_pair<T, true>(w0, fk[h]),
                           code_pair<T, false>(w1, fk[h]), code_pair<T, true>(w1, fk[h])};
            } else {
              kf = t.k[h][kb];
            }
            if (A::kForm && !WHOLE && W::depth(kb, g) >= a.D) kf = u32x4_t{0u, 0u, 0u, 0u};
            acc = mfma16<T>(kf, qf[q][kb], acc);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = A::kForm ? acc[i] : product(acc[i], a.scale);
            if (LW && !A::kForm) v = t.w[h][i] == -INFINITY ? -INFINITY : v + t.w[h][i];  // (whatever the key is)
            s[4 * h + i] = v;
          }
        }
        if constexpr (A::kForm) {
          if (a.cap > 0.f) {
            cap_scores<8, LW>(s, a.scale, a.cap);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = product(s[j], a.scale);
          }
          if (a.slopes) {
            const int at = c_of[q] - k - 4 * g;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[j] = fmaf(-slope[q], fabsf((float)(at - (j < 4 ? 0 : 16) - (j & 3))), s[j]);
          }
          if (LW) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[j] = t.w[j >> 2][j & 3] == -INFINITY ? -INFINITY : s[j] + t.w[j >> 2][j & 3];  // (whatever the key is)
          }
        }
        if (!all) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = k + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
            const bool see = (j < 4 ? t.ok[0] : t.ok[1]) && sees(q, key);
            s[j] = see ? s[j] : -INFINITY;
          }
        }
        float mx = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
        mx = max16(max32(mx));
        const float mn = fmaxf(m_[q], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float al = factor<LW>(m_[q], ms);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[j] = term<T, LW>(s[j], ms);
          sum += s[j];
        }
        m_[q] = mn;
        l_[q] = l_[q] * al + sum;
#pragma unroll
        for (int e = 0; e < DV; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[q][e][i] *= al;
#pragma unroll
        for (int j = 0; j < 4; ++j) pf[q][j] = T::pack(s[2 * j], s[2 * j + 1]);
      }
      auto multiply = [&](const uint32_t(&v)[8][W::VW]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < DV; ++e) {
          u32x4_t vf;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vf[j] = __builtin_amdgcn_perm(v[2 * j + 1][e / 2], v[2 * j][e / 2], e & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int q = 0; q < NQ; ++q) o[q][e] = mfma16<T>(vf, pf[q], o[q][e]);
        }
      };
      if constexpr (!F8) {
        multiply(t.v);
      } else if (!all) {
        uint32_t v[8][W::VW];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int i = 0; i < W::VW / 2; ++i) {
            v[j][2 * i] = code_pair<T, false>(t.v[j][i], fv[j / 4]);
            v[j][2 * i + 1] = code_pair<T, true>(t.v[j][i], fv[j / 4]);
          }
        }
        clean(v, t, k, false);
        multiply(v);
      } else {
        // codes are paired before they are widened: half the permutes
        if (LW) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < DP / 64; ++i)
              if (t.w[j >> 2][j & 3] == -INFINITY) t.v[j][i] = 0u;
#pragma unroll
          for (int h = 0; h < 2; ++h)  // (zeros stay zeros in a block whose scale is NaN)
            if (fmaxf(fmaxf(t.w[h][0], t.w[h][1]), fmaxf(t.w[h][2], t.w[h][3])) == -INFINITY) fv[h] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < DV; e += 2) {
          u32x4_t v0, v1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = __builtin_amdgcn_perm(t.v[2 * j + 1][e / 4], t.v[2 * j][e / 4],
                                                     e & 2 ? 0x07030602u : 0x05010400u);
            v0[j] = code_pair<T, false>(w, fv[j / 2]);
            v1[j] = code_pair<T, true>(w, fv[j / 2]);
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            o[q][e] = mfma16<T>(v0, pf[q], o[q][e]);
            o[q][e + 1] = mfma16<T>(v1, pf[q], o[q][e + 1]);
          }
        }
      }
    };

    int k = k0 + 32 * wave;
    Pages pg = pages_of(a, row, slot_of(k));
    if constexpr (A::kForm && STAGES == 2) {
      if (k < k1) {
        // loads a step ahead, behind the last step few bytes of it again
        Tile<DP, LW, F8> t[2];
        const int last = k + (k1 - 1 - k) / kDecodeUnit * kDecodeUnit;
        auto ahead = [&](int n) __attribute__((always_inline)) { return min(k + n * kDecodeUnit, last); };
        auto fetch = [&](int n, Tile<DP, LW, F8>& to) __attribute__((always_inline)) {
          W::load(a, pg, head, slot_of(ahead(n)), k + n * kDecodeUnit < k1 ? lane : -1, to);
          pg = pages_of(a, row, slot_of(ahead(n + 1)));
        };
        fetch(0, t[0]);
        auto step = [&](int i) __attribute__((always_inline)) {
          fetch(1, t[i ^ 1]);
          process(t[i], slot_of(k));
          k += kDecodeUnit;
          return k < k1;
        };
        for (;;) {
          if (!step(0)) break;
          if (!step(1)) break;
        }
      }
    } else if constexpr (STAGES == 2) {
      if (k < k1) {
        Tile<DP, LW, F8> ta, tb;
        W::load(a, pg, head, slot_of(k), lane, ta);
        pg = pages_of(a, row, slot_of(k + kDecodeUnit));
        for (;;) {
          if (k + kDecodeUnit < k1) W::load(a, pg, head, slot_of(k + kDecodeUnit), lane, tb);
          pg = pages_of(a, row, slot_of(k + 2 * kDecodeUnit));
          process(ta, slot_of(k));
          k += kDecodeUnit;
          if (k >= k1) break;
          if (k + kDecodeUnit < k1) W::load(a, pg, head, slot_of(k + kDecodeUnit), lane, ta);
          pg = pages_of(a, row, slot_of(k + 2 * kDecodeUnit));
          process(tb, slot_of(k));
          k += kDecodeUnit;
          if (k >= k1) break;
        }
      }
    } else {
      for (; k < k1; k += kDecodeUnit) {
        Tile<DP, LW, F8> t;
        W::load(a, pg, head, slot_of(k), lane, t);
        pg = pages_of(a, row, slot_of(k + kDecodeUnit));
        process(t, slot_of(k));
      }
    }

    if (some_odd) {
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        if ((k / 32) % 4 != wave) continue;  // (another wavefront's)
        const int key = slot_of(k), kt = key - key % 32;
        const Pages held = pages_of(a, row, kt);
        if (all_see(kt) && held.ok[0] && held.ok[1]) continue;  // (nothing was taken out)
        bool ok;
        const int page = page_of_uniform(a, row, key, ok), off = key & ((1 << a.page_shift) - 1);
        if (!ok || (LW && a.lw[page * a.lw_page + head * a.lw_head + off] == -INFINITY)) continue;
        const uint8_t* vp = a.v + page * a.v_page + off * a.v_slot + head * a.v_head;
        float scale = 0.f;
        if constexpr (F8) scale = block_scale(a.vs[page * a.vs_page + head * a.vs_head + (off >> 4)]);
#pragma unroll
        for (int e = 0; e < DV; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = W::column(4 * g + i, e);
            uint32_t v = 0u;
            if constexpr (F8)
              v = d < a.D ? code_pair<T, false>(vp[d], scale) & 0xffffu : 0u;
            else
              v = d < a.D ? ((const uint16_t*)vp)[d] : 0u;
            if ((v & T::kExp) == T::kExp) {
#pragma unroll
              for (int q = 0; q < NQ; ++q)
                if (sees(q, key)) o[q][e][i] += T::lo(v);
            }
          }
      }
    }

    // Join the four wavefronts.
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const float l = sum16(sum32(l_[q]));
      if (g == 0) {
        s_ml[wave][16 * q + x][0] = m_[q];
        s_ml[wave][16 * q + x][1] = l;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < DV; e += 4)
          *(f32x4_t*)&s_o[wave][16 * q + x][W::column(4 * g + i, e)] =
              f32x4_t{o[q][e][i], o[q][e + 1][i], o[q][e + 2][i], o[q][e + 3][i]};
    }
    __syncthreads();
    constexpr int PR = DP / 4;  // 16-byte pieces of a row
    for (int p = tid; p < BM * PR; p += kWgThreads) {
      const int m = p / PR, d = (p - m * PR) * 4;
      if (m >= rows) break;
      float M = fmaxf(fmaxf(s_ml[0][m][0], s_ml[1][m][0]), fmaxf(s_ml[2][m][0], s_ml[3][m][0]));
      const float ms = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = factor<LW>(s_ml[v][m][0], ms);
        L += f * s_ml[v][m][1];
        const f32x4_t ov = *(const f32x4_t*)&s_o[v][m][d];
        if (s_ml[v][m][0] != -INFINITY) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] += f * ov[i];
        }
      }
      if (whole) {
        const int i = m / a.G, hq = head * a.G + (m - i * a.G);
        const int64_t tok = w.q.q0 + i;
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        if (d < a.D)
          *(u32x2_t*)(a.out + tok * a.o_token + hq * a.o_head + d) =
              u32x2_t{T::pack(acc[0] * inv, acc[1] * inv), T::pack(acc[2] * inv, acc[3] * inv)};
        if (a.lse && d == 0) a.lse[tok * a.Hq + hq] = log_sum<T, LW>(ms, L);
      } else {
        const int64_t at = (int64_t)part * BM + m;
        *(f32x4_t*)(a.part_o + at * DP + d) = acc;
        if (d == 0) a.part_ml[at] = f32x2_t{M, L};
      }
    }
    pos += len;
    if (pos >= line.upto) break;
    w.q = next_request<BM, kDecodeUnit>(a, w.r, w.head);
    w.off = 0;
    __syncthreads();  // (s_ml and s_o are read)
  }
}

}  // namespace
}  // namespace kmkv

// Attention of few rows (at most 16 or 32 for each request and cache head)
// over a paged cache: the decode step, and the join of divided rows.
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

// One step's keys and values of a wavefront: 32 keys.
template <int DP, bool LW>
struct Tile {
  u32x4_t k[2][DP / 32];
  uint32_t v[8][DP / 32];  // 8 keys x DP / 16 columns
  f32x4_t w[LW ? 2 : 1];
  bool ok[2];              // (uniform) the halves' pages are in the cache
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
template <class T, int DP, int NQ, bool LW, bool WHOLE>
struct Decode {
  static constexpr int BM = 16 * NQ, KB = DP / 32, DV = DP / 16, VW = DP / 32;
  static constexpr int LS = DP + 4;  // LDS row of a wavefront's partial result, in floats
  // Neighbouring columns of a lane: one load, whose 16 lanes read whole rows of up to 128 columns.
  static constexpr int kRun = DV < 8 ? DV : 8;
  // The e-th column that lane x of a group loads.
  static __device__ __forceinline__ constexpr int column(int x, int e) {
    return e / kRun * (16 * kRun) + x * kRun + e % kRun;
  }

  static __device__ __forceinline__ void load(const AttendArgs& a, const Pages& pg, int head, int k, int lane,
                                              Tile<DP, LW>& t) {
    const int x = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k + 16 * h;
      t.ok[h] = pg.ok[h];
      const int64_t page = pg.page[h];
      const int off = key & ((1 << a.page_shift) - 1);
      const uint8_t* kp = a.k + page * a.k_page + off * a.k_slot + head * a.k_head + (x * a.k_slot + g * 16);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (WHOLE || kb * 32 + g * 8 < a.D)
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
          if (WHOLE || column(x, 0) < a.D) w = __builtin_nontemporal_load((const u32x2_t*)s);
          d[0] = w[0];
          d[1] = w[1];
        } else {
#pragma unroll
          for (int c = 0; c < VW; c += 4) {
            u32x4_t w = {0u, 0u, 0u, 0u};
            if (WHOLE || column(x, 2 * c) < a.D)
              w = __builtin_nontemporal_load((const u32x4_t*)(s + column(0, 2 * c) * 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) d[c + i] = w[i];
          }
        }
      }
    }
  }
};

template <class T, int DP, int NQ, bool LW, bool WHOLE>
__global__ __launch_bounds__(kWgThreads, decode_per_cu(DP, 16 * NQ)) void decode_kernel(AttendArgs a) {
  using W = Decode<T, DP, NQ, LW, WHOLE>;
  constexpr int BM = W::BM, KB = W::KB, DV = W::DV, LS = W::LS;
  constexpr bool PF = DP <= 128;  // (two steps' registers)
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
    int k0, k1;
    key_range<kDecodeUnit>(a, w.q, 0, w.q.n - 1, w.off, len, k0, k1);
    const int32_t* row = a.table + w.r * a.table_stride;

    // queries: this lane's column of each group of 16 rows
    u32x4_t qf[NQ][KB];
    int jmin[NQ], jmax[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int m = min(16 * q + x, rows - 1);
      const int i = m / a.G, hq = head * a.G + (m - i * a.G);
      const uint16_t* qp = a.q + (int64_t)(w.q.q0 + i) * a.q_token + hq * a.q_head + g * 8;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        qf[q][kb] = u32x4_t{0u, 0u, 0u, 0u};
        if (kb * 32 + g * 8 < a.D) qf[q][kb] = *(const u32x4_t*)(qp + kb * 32);
      }
      jmax[q] = min(c + i, k1 - 1);
      jmin[q] = a.window > 0 ? c + i - a.window + 1 : 0;
    }
    // a step whose keys all rows see: from `full0`, up to `full1`
    const int full1 = min(c + 1, k1), full0 = a.window > 0 ? c + w.q.n - a.window : 0;

    f32x4_t o[NQ][DV];
    float m_[NQ], l_[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m_[q] = -INFINITY;
      l_[q] = 0.f;
#pragma unroll
      for (int e = 0; e < DV; ++e) o[q][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    bool some_odd = false;
    auto process = [&](Tile<DP, LW>& t, int k) __attribute__((always_inline)) {
      const bool all = k >= full0 && k + 32 <= full1 && t.ok[0] && t.ok[1];
      bool odd = false;
      if (!all || LW) {
        // values of keys that no row sees are taken out, whatever they are
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = k + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
          bool in = (j < 4 ? t.ok[0] : t.ok[1]) && key < k1;
          if (LW) in = in && t.w[j >> 2][j & 3] != -INFINITY;
#pragma unroll
          for (int i = 0; i < W::VW; ++i) {
            if (!in) t.v[j][i] = 0u;
            if (!all) odd |= odd_pair<T>(t.v[j][i]);
          }
        }
        // rows differ in what they see and a value is infinite or NaN: take it
        // out of the product and add it in the end to the rows that see it
        if (__any(odd)) {
          some_odd = true;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < W::VW; ++i) t.v[j][i] = even_pair<T>(t.v[j][i]);
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
          for (int kb = 0; kb < KB; ++kb) acc = mfma16<T>(t.k[h][kb], qf[q][kb], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = product(acc[i], a.scale);
            if (LW) v = t.w[h][i] == -INFINITY ? -INFINITY : v + t.w[h][i];  // (whatever the key is)
            s[4 * h + i] = v;
          }
        }
        if (!all) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = k + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
            const bool see = (j < 4 ? t.ok[0] : t.ok[1]) && key >= jmin[q] && key <= jmax[q];
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
#pragma unroll
      for (int e = 0; e < DV; ++e) {
        u32x4_t vf;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          vf[j] = __builtin_amdgcn_perm(t.v[2 * j + 1][e / 2], t.v[2 * j][e / 2], e & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int q = 0; q < NQ; ++q) o[q][e] = mfma16<T>(vf, pf[q], o[q][e]);
      }
    };

    int k = k0 + 32 * wave;
    Pages pg = pages_of(a, row, k);
    if constexpr (PF) {
      if (k < k1) {
        Tile<DP, LW> ta, tb;
        W::load(a, pg, head, k, lane, ta);
        pg = pages_of(a, row, k + kDecodeUnit);
        for (;;) {
          if (k + kDecodeUnit < k1) W::load(a, pg, head, k + kDecodeUnit, lane, tb);
          pg = pages_of(a, row, k + 2 * kDecodeUnit);
          process(ta, k);
          k += kDecodeUnit;
          if (k >= k1) break;
          if (k + kDecodeUnit < k1) W::load(a, pg, head, k + kDecodeUnit, lane, ta);
          pg = pages_of(a, row, k + 2 * kDecodeUnit);
          process(tb, k);
          k += kDecodeUnit;
          if (k >= k1) break;
        }
      }
    } else {
      for (; k < k1; k += kDecodeUnit) {
        Tile<DP, LW> t;
        W::load(a, pg, head, k, lane, t);
        pg = pages_of(a, row, k + kDecodeUnit);
        process(t, k);
      }
    }

    if (some_odd) {
#pragma unroll 1
      for (int key = k0; key < k1; ++key) {
        const int kt = key - key % 32;
        if ((kt / 32) % 4 != wave) continue;  // (another wavefront's)
        const Pages held = pages_of(a, row, kt);
        if (kt >= full0 && kt + 32 <= full1 && held.ok[0] && held.ok[1]) continue;  // (nothing was taken out)
        bool ok;
        const int page = page_of_uniform(a, row, key, ok), off = key & ((1 << a.page_shift) - 1);
        if (!ok || (LW && a.lw[page * a.lw_page + head * a.lw_head + off] == -INFINITY)) continue;
        const uint16_t* vp = (const uint16_t*)(a.v + page * a.v_page + off * a.v_slot + head * a.v_head);
#pragma unroll
        for (int e = 0; e < DV; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = W::column(4 * g + i, e);
            const uint32_t v = d < a.D ? vp[d] : 0u;
            if ((v & T::kExp) == T::kExp) {
#pragma unroll
              for (int q = 0; q < NQ; ++q)
                if (key >= jmin[q] && key <= jmax[q]) o[q][e][i] += T::lo(v);
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

// out = sum over the parts of e^(m - M) o, divided by that of l.  One thread
// takes 4 columns of a row in every NG-th part, four parts at a time; NG such
// threads are joined through LDS.
template <class T, int DP, bool LW, int NG>
__global__ __launch_bounds__(kWgThreads) void join_kernel(JoinArgs a) {
  constexpr int PR = DP / 4, ROWS = kWgThreads / (PR * NG);
  __shared__ __align__(16) float s_o[NG > 1 ? NG : 1][NG > 1 ? ROWS * PR : 1][4];
  __shared__ float s_ml[NG > 1 ? NG : 1][NG > 1 ? ROWS : 1][2];
  const int t = blockIdx.x, total = a.query_start[a.R];
  const int4 f = a.info[t];
  if (t >= total) return;
  const int p = threadIdx.x % (PR * ROWS), ng = threadIdx.x / (PR * ROWS);
  const int hq = blockIdx.y * ROWS + p / PR, d = (p % PR) * 4;
  const int head = min(hq, a.Hq - 1) / a.G;
  const int64_t m = (int64_t)f.z * a.G + (min(hq, a.Hq - 1) - head * a.G);  // row of the request
  // the parts: n of them, the first at row `at`, the others from row `at1` on every `step` rows
  const float* po;
  const f32x2_t* pml;
  int n;
  int64_t at, at1, step;
  if (f.w & 1) {  // chunk launch
    n = f.y;
    if (n <= 1) return;
    const int64_t tile = m / kChunkRows, first = f.x + tile * n;
    if (f.x < 0 || f.z < 0 || first + n > a.parts1) return;  // (no such part: more new tokens than max_new)
    po = a.o1;
    pml = a.ml1;
    step = (int64_t)a.Hkv * kChunkRows;
    at = (first * a.Hkv + head) * kChunkRows + (m - tile * kChunkRows);
    at1 = at + step;
  } else {  // decode launch: the pieces that the request's units of this head lie in
    const int64_t per_head = *a.per_head, all = per_head * a.Hkv;
    const int64_t p0 = head * per_head + (((int64_t)(f.w >> 1) << 32) | (uint32_t)f.x), p1 = p0 + f.y;
    if (f.y < 1 || m < 0 || m >= a.bm0 || p0 < 0 || p1 > all) return;  // (no such part: more new tokens than max_new)
    const int64_t pieces = a.pieces < all ? a.pieces : all;
    const int64_t w0 = piece_of(p0, all, pieces), w1 = piece_of(p1 - 1, all, pieces);
    n = (int)(w1 - w0) + 1;
    if (n <= 1) return;
    po = a.o0;
    pml = a.ml0;
    step = 2 * a.bm0;
    at1 = 2 * (w0 + 1) * a.bm0 + m;  // a piece's first part
    at = at1 - step + (p0 > piece_start(w0, all, pieces) ? a.bm0 : 0);  // ... its last
  }
  float M = -INFINITY, L = 0.f;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = ng; s0 < n; s0 += 4 * NG) {
    f32x2_t ml[4];
    f32x4_t ov[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = min(s0 + j * NG, n - 1);  // (the last part again, with no weight)
      const int64_t e = s == 0 ? at : at1 + (s - 1) * step;
      ml[j] = pml[e];
      ov[j] = *(const f32x4_t*)(po + e * DP + d);
      if (s0 + j * NG >= n) ml[j] = f32x2_t{-INFINITY, 0.f};
    }
    const float mn = fmaxf(fmaxf(fmaxf(ml[0][0], ml[1][0]), fmaxf(ml[2][0], ml[3][0])), M);
    const float ms = mn == -INFINITY ? 0.f : mn, al = factor<LW>(M, ms);
    M = mn;
    L *= al;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= al;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w = factor<LW>(ml[j][0], ms);
      L += w * ml[j][1];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ml[j][0] != -INFINITY) acc[i] += w * ov[j][i];  // (a part that saw nothing wrote no o)
    }
  }
  if constexpr (NG > 1) {
    *(f32x4_t*)s_o[ng][p] = acc;
    if (d == 0) {
      s_ml[ng][p / PR][0] = M;
      s_ml[ng][p / PR][1] = L;
    }
    __syncthreads();
    if (ng > 0) return;
#pragma unroll
    for (int g = 1; g < NG; ++g) M = fmaxf(M, s_ml[g][p / PR][0]);
    const float ms = M == -INFINITY ? 0.f : M;
    L = 0.f;
    acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float w = factor<LW>(s_ml[g][p / PR][0], ms);
      L += w * s_ml[g][p / PR][1];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += w * s_o[g][p][i];
    }
  }
  if (hq >= a.Hq || d >= a.D) return;
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  *(u32x2_t*)(a.out + t * a.o_token + hq * a.o_head + d) =
      u32x2_t{T::pack(acc[0] * inv, acc[1] * inv), T::pack(acc[2] * inv, acc[3] * inv)};
  if (a.lse && d == 0) a.lse[(int64_t)t * a.Hq + hq] = log_sum<T, LW>(M == -INFINITY ? 0.f : M, L);
}

template <class T, int DP, int NQ, bool LW>
void decode_whole(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.pieces);
  if (a.D == DP)
    decode_kernel<T, DP, NQ, LW, true><<<grid, kWgThreads, 0, stream>>>(a);
  else
    decode_kernel<T, DP, NQ, LW, false><<<grid, kWgThreads, 0, stream>>>(a);
}

template <class T, int DP, int NQ>
void decode_lw(const AttendArgs& a, hipStream_t stream) {
  if (a.lw)
    decode_whole<T, DP, NQ, true>(a, stream);
  else
    decode_whole<T, DP, NQ, false>(a, stream);
}

template <class T, int NQ>
void decode_dim(const AttendArgs& a, hipStream_t stream) {
  const int dp = dim_pad(a.D);
  if (dp == 64)
    decode_lw<T, 64, NQ>(a, stream);
  else if (dp == 128)
    decode_lw<T, 128, NQ>(a, stream);
  else
    decode_lw<T, 256, NQ>(a, stream);
}

template <class T, int DP, bool LW>
void join_rows(const JoinArgs& a, hipStream_t stream) {
  // Few rows can have many parts each (as many as there are workgroups to
  // share among them): 8 threads share them.  Many rows have few parts or
  // none.  (Measured, whole calls: 56 rows of 146 parts 87 us with 8 threads,
  // 99 with one; 4,064 rows of 4 parts 143 us with 8, 139 with one; 16,352
  // rows of one or two 178 against 163.)
  constexpr int NG = DP == 256 ? 4 : 8;
  constexpr int kFewRows = 1024;
  if ((int64_t)a.T * a.Hq <= kFewRows) {
    constexpr int rows = kWgThreads / (DP / 4 * NG);
    join_kernel<T, DP, LW, NG><<<dim3((unsigned)a.T, (unsigned)((a.Hq + rows - 1) / rows)), kWgThreads, 0, stream>>>(a);
  } else {
    constexpr int rows = kWgThreads / (DP / 4);
    join_kernel<T, DP, LW, 1><<<dim3((unsigned)a.T, (unsigned)((a.Hq + rows - 1) / rows)), kWgThreads, 0, stream>>>(a);
  }
}

template <class T, bool LW>
void join_dim(const JoinArgs& a, hipStream_t stream) {
  const int dp = dim_pad(a.D);
  if (dp == 64)
    join_rows<T, 64, LW>(a, stream);
  else if (dp == 128)
    join_rows<T, 128, LW>(a, stream);
  else
    join_rows<T, 256, LW>(a, stream);
}

}  // namespace

hipError_t launch_decode(const AttendArgs& a, int dt, int bm, hipStream_t stream) {
  if (dt == 1)
    bm == 16 ? decode_dim<BF16, 1>(a, stream) : decode_dim<BF16, 2>(a, stream);
  else
    bm == 16 ? decode_dim<F16, 1>(a, stream) : decode_dim<F16, 2>(a, stream);
  return hipGetLastError();
}

hipError_t launch_join(const JoinArgs& a, int dt, hipStream_t stream) {
  if (dt == 1)
    a.weighted ? join_dim<BF16, true>(a, stream) : join_dim<BF16, false>(a, stream);
  else
    a.weighted ? join_dim<F16, true>(a, stream) : join_dim<F16, false>(a, stream);
  return hipGetLastError();
}

}  // namespace kmkv

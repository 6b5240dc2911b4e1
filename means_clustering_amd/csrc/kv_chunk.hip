// Attention of many rows of each request over a paged cache: chunks of a
// prompt.  The same sums as the decode kernel,
//
//   s = scale * (K q) + weight,  m = running maximum, p = e^(s - m),
//   l = sum p,  o = sum p v,  out = o / l,
//
// bound by the matrix cores.  A workgroup takes 128 rows, 32 for each
// wavefront, and walks its keys in tiles of BN, staged through LDS for all
// four wavefronts: the next tile is loaded into registers while this one is
// multiplied, and stored to the other LDS buffer after.
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
// or with the row, so that the reads of K (8 rows, one piece column) and of V
// (4 rows, 2 neighbouring pieces) meet no bank twice.
#include "kv_attend.hpp"

namespace kmkv {
namespace {

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
  constexpr int KB = DP / 16;              // depth steps of K Q'
  constexpr int CH = DP / 8;               // 16-byte pieces of an LDS row
  constexpr int RP = kWgThreads / CH;      // rows staged by one round of the workgroup
  constexpr int ROUNDS = BN / RP;
  constexpr int NT = BN / 32, DT = DP / 32;
  __shared__ int64_t scratch[16];
  __shared__ __align__(16) u32x4_t s_k[2][BN * CH];
  __shared__ __align__(16) u32x4_t s_v[2][BN * CH];
  __shared__ __align__(16) float s_w[2][LW ? BN : 4];
  // first key of the buffer's tile if it holds an infinite or NaN value (taken out), or lies partly in no page
  __shared__ int s_odd[2], s_bad[2];
  const int head = blockIdx.x % a.Hkv, it = blockIdx.x / a.Hkv;
  Item w;
  if (!find_item<BM, BN>(a, it, w, scratch)) return;
  const int tid = threadIdx.x, lane = tid & 63, x = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = w.q.n * a.G, c = w.q.c;
  const int tok0 = w.tile * BM / a.G, tok1 = min((w.tile * BM + BM - 1) / a.G, w.q.n - 1);
  if (head == 0 && w.split == 0)
    for (int i = tok0 + tid; i <= tok1; i += kWgThreads) a.info[w.q.q0 + i] = make_int4(w.part0, w.splits, i, 1);
  int k0, k1;
  key_range<BM, BN>(a, w, k0, k1);
  const int32_t* row = a.table + w.r * a.table_stride;

  // this lane's query row
  const int m = w.tile * BM + 32 * wave + x, mc = min(m, rows - 1);
  const int qi = mc / a.G, hq = head * a.G + (mc - qi * a.G);
  u32x4_t qf[KB];
  {
    const uint16_t* qp = a.q + (int64_t)(w.q.q0 + qi) * a.q_token + hq * a.q_head + 8 * h;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      qf[kb] = u32x4_t{0u, 0u, 0u, 0u};
      if (16 * kb + 8 * h < a.D) qf[kb] = *(const u32x4_t*)(qp + 16 * kb);
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

  // staging: this thread's piece of a row, ROUNDS rows
  const int sc = tid % CH, sr = tid / CH;
  u32x4_t rk[ROUNDS], rv[ROUNDS];
  bool rok[ROUNDS];
  float rw = 0.f;
  bool bad = false;
  auto load = [&](int kt) {
    bad = false;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      // a wavefront's rows of a round lie in one page
      const int key0 = __builtin_amdgcn_readfirstlane(kt + i * RP + (wave * 64) / CH);
      bool ok;
      const int page = page_of(a, row, key0, ok);
      const int key = kt + i * RP + sr, off = key & ((1 << a.page_shift) - 1);
      rok[i] = ok && key < k1;
      bad |= !ok && key0 < k1;
      rk[i] = rv[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (8 * sc < a.D) {
        rk[i] = *(const u32x4_t*)(a.k + page * a.k_page + head * a.k_head + (off * a.k_slot + sc * 16));
        rv[i] = *(const u32x4_t*)(a.v + page * a.v_page + head * a.v_head + (off * a.v_slot + sc * 16));
      }
      if (LW) {
        const float lw = a.lw[page * a.lw_page + head * a.lw_head + off];
        rok[i] = rok[i] && lw != -INFINITY;
      }
    }
    if (LW && tid < BN) {
      bool ok;
      const int page = page_of(a, row, kt + tid, ok);
      rw = ok ? a.lw[page * a.lw_page + head * a.lw_head + ((kt + tid) & ((1 << a.page_shift) - 1))] : -INFINITY;
    }
  };
  auto store = [&](int kt, int buf) {
    const bool part = kt < wfull0 || kt + BN > wfull1;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // values (and, for the sake of their products, keys) that no row sees are taken out, whatever they are
        if (!rok[i]) rk[i][j] = rv[i][j] = 0u;
        if (part) odd |= odd_pair<T>(rv[i][j]);
      }
    }
    if (part && __any(odd)) {
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) rv[i][j] = even_pair<T>(rv[i][j]);
      if (lane == 0) s_odd[buf] = kt;
    }
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int r = i * RP + sr;
      s_k[buf][r * CH + (sc ^ (r & 7))] = rk[i];
      s_v[buf][r * CH + (sc ^ ((2 * r) & (CH - 1) & 14))] = rv[i];
    }
    if (bad && lane == 0) s_bad[buf] = kt;
    if (LW && tid < BN) s_w[buf][tid] = rw;
  };

  if (tid < 2) s_odd[tid] = s_bad[tid] = -1;
  __syncthreads();
  if (k0 < k1) {
    load(k0);
    store(k0, 0);
  }
  __syncthreads();
  int buf = 0;
  for (int kt = k0; kt < k1; kt += BN, buf ^= 1) {
    const bool more = kt + BN < k1;
    if (more) load(kt + BN);
    if (kt + BN > see0 && kt < see1) {
      f32x16_t s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int r = 32 * t + x;
          s[t] = mfma32<T>(s_k[buf][r * CH + ((2 * kb + h) ^ (r & 7))], qf[kb], s[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          f32x4_t wv;
          if (LW) wv = *(const f32x4_t*)&s_w[buf][32 * t + 8 * b + 4 * h];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = s[t][4 * b + i] * a.scale;
            if (LW) v = wv[i] == -INFINITY ? -INFINITY : v + wv[i];
            s[t][4 * b + i] = v;
          }
        }
      const bool holes = s_bad[buf] == kt;
      if (kt < full0 || kt + BN > full1 || holes) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = kt + 32 * t + 8 * (i / 4) + 4 * h + (i & 3);
            bool see = key >= jmin && key <= jmax;
            if (holes && see) (void)page_of(a, row, key, see);
            s[t][i] = see ? s[t][i] : -INFINITY;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
      mx = max32(mx);
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
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[t][i] = factor<LW>(s[t][i], ms);
          sum += s[t][i];
        }
      l_ += sum;
#pragma unroll
      for (int u = 0; u < 2 * NT; ++u) {
        u32x4_t pf;
#pragma unroll
        for (int j = 0; j < 4; ++j) pf[j] = T::pack(s[u / 2][8 * (u & 1) + 2 * j], s[u / 2][8 * (u & 1) + 2 * j + 1]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const int r = 16 * u + 4 * h + ((lane & 15) >> 2);
          const int col = 32 * d + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);  // elements
          u32x4_t vf;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int re = r + 8 * e;
            const char* at = (const char*)&s_v[buf][re * CH + ((col >> 3) ^ ((2 * re) & (CH - 1) & 14))] + (col & 4) * 2;
            const s16x4_t tr = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4_t*)(__attribute__((address_space(3))) char*)at);
            const u32x2_t two = __builtin_bit_cast(u32x2_t, tr);
            vf[2 * e] = two[0];
            vf[2 * e + 1] = two[1];
          }
          o[d] = mfma32<T>(vf, pf, o[d]);
        }
      }
      if (s_odd[buf] == kt) {
#pragma unroll 1
        for (int key = kt; key < min(kt + BN, k1); ++key) {
          bool ok;
          const int page = page_of(a, row, key, ok);
          const int off = key & ((1 << a.page_shift) - 1);
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
    }
    if (more) store(kt + BN, buf ^ 1);
    __syncthreads();
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
    if (a.lse && h == 0) a.lse[tok * a.Hq + hq] = log_sum<LW>(ms, L);
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

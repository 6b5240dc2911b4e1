// The append with several position axes, and into an 8-bit cache; and what an
// 8-bit cache holds, read back.
//
//   y = x / sqrt(mean(x^2) + eps) * weight,  (a, b) -> (a c - b s, b c + a s),
//   pair i by the position on axis[i]
//
// as in kv_append.hip, rows in fp32 and rounded once.  An 8-bit cache has one
// scale 2^e for each block of 16 slots of a page and head.  A = the largest
// finite |y| that the call writes into the block, and
//
//   need = the least e >= -126 with A <= 448 * 2^e   (448 is e4m3's largest)
//   e    = need, if the block's first slot is written, else max(old e, need)
//   code = e4m3(y * 2^-e),  older codes of the block: e4m3(code * 2^(old - e))
//
// Scales are powers of two, so y * 2^-e is exact, older codes move without a
// rounding (but for those that become subnormal), and the attention's
// conversion takes the scale at no cost; e4m3 rounds to 4 bits whatever the
// scale is, so nothing is lost against other scales.
//
// A workgroup takes as many tokens as it has groups of lanes, for one or two
// heads of the keys or of the values.  A group makes its token's row and keeps it
// in registers; rows of blocks that reach over the window's ends are made beside
// it, for their A only.  The rows' maxima meet in LDS, each group takes those of
// its block's tokens (at most 15 places away), and writes its row; the group of
// the block's first token writes the scale.  Two workgroups may so work out the
// scale of one block, each for its own tokens, and have to agree: what makes a row
// is fused by hand or not at all (norm(), turn()), so its copies round alike.
// Queries (and with a 16-bit cache all rows) are rows on their own, as in
// kv_append.hip.
//
// Measured (bf16, 8 cache heads of 128): 16,001 tokens 46 us for keys and values
// (98 MB, 22 us at a copy's rate) and 57 us for 32 heads of queries (HBM); what
// holds up the former is the way from a row's load through norm, angles and the
// block's maximum to its store, with vector units busy half of the time.  33 tokens
// 5.3 us, a launch and four dependent loads.  8,191 tokens of 28 + 4 + 4 heads by 3
// axes into 16 bits 28.5 us (5.4 TB/s).
//   * A wavefront for each block, which looks for its tokens among 63 others and
//     gathers their rows: 135 us for 16,001 tokens with their read, 122 by windows.
//   * A token's slot and positions loaded once, not for each row's angles: 51 us
//     against 37 for 8,191 tokens with axes (whole calls).
//   * Queries in the writers' launch hold twice the registers that they need:
//     106 us against 100 in two launches.
#include <type_traits>

#include "kv_rows.hpp"

namespace kmkv {
namespace {

constexpr float kLargest = 3.402823466e38f;

// A token's slot and positions (the axes that there are; 0 beyond), and whether
// it is none of padding.
constexpr int kAxes = 4;
struct Where {
  int slot, pos[kAxes];
  bool live;
};
__device__ __forceinline__ Where where(const FormAppendArgs& a, int t) {
  Where w;
  w.slot = a.slots ? a.slots[t] : t;
#pragma unroll
  for (int i = 0; i < kAxes; ++i) w.pos[i] = i < a.axes ? a.positions[i * a.axis_stride + t] : 0;
  w.live = w.slot >= 0 && w.slot < a.num_slots;
#pragma unroll
  for (int i = 0; i < kAxes; ++i) w.live = w.live && w.pos[i] >= 0 && w.pos[i] < a.max_pos;
  return w;
}

// This lane's two chunks of 8 elements of a row.
template <bool PAIRS>
struct Lane {
  int u, c0, c1;
  bool mine, turn;
  __device__ __forceinline__ Lane(const FormAppendArgs& a, int u_) : u(u_) {
    const int half = a.rot / 16;  // chunks of half the rotated part
    if (PAIRS) {
      c0 = 2 * u;
      c1 = c0 + 1;
      turn = c0 * 8 < a.rot;
    } else {
      turn = u < half;
      c0 = turn ? u : 2 * u;
      c1 = turn ? u + half : c0 + 1;
    }
    mine = u * 16 < a.D;
  }
};

// Joins the values of the LPR lanes of a row, all in registers: neighbours,
// pairs, then mirrored halves.
template <int LPR, class V, class Op>
__device__ __forceinline__ V join_lanes(V v, Op op) {
  auto moved = [&](auto c) __attribute__((always_inline)) {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(c)::value, 0xf, 0xf, false));
  };
  v = op(v, moved(std::integral_constant<int, 0xb1>{}));
  if (LPR > 2) v = op(v, moved(std::integral_constant<int, 0x4e>{}));
  if (LPR > 4) v = op(v, moved(std::integral_constant<int, 0x141>{}));
  if (LPR > 8) v = op(v, moved(std::integral_constant<int, 0x140>{}));
  return v;
}

template <int LPR, bool PAIRS>
__device__ __forceinline__ void norm(const FormAppendArgs& a, const Lane<PAIRS>& l, const float* weight, float* x) {
#pragma clang fp contract(off)
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) ss += __shfl_xor(ss, d);
  const float inv = 1.0f / sqrtf(ss / (float)a.D + a.eps);
  if (!l.mine) return;
  const f32x4_t g0 = *(const f32x4_t*)(weight + l.c0 * 8), g1 = *(const f32x4_t*)(weight + l.c0 * 8 + 4);
  const f32x4_t g2 = *(const f32x4_t*)(weight + l.c1 * 8), g3 = *(const f32x4_t*)(weight + l.c1 * 8 + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] *= inv * g0[i];
    x[4 + i] *= inv * g1[i];
    x[8 + i] *= inv * g2[i];
    x[12 + i] *= inv * g3[i];
  }
}

// Cosines and sines of this lane's 8 pairs for a live token: those of chunk u's
// pairs (halves), or of the pairs in both chunks (interleaved).  axis: of the 8
// pairs, a byte each.
struct Angles {
  float c[8], s[8];
};
template <bool PAIRS>
__device__ __forceinline__ uint64_t axes_of(const FormAppendArgs& a, const Lane<PAIRS>& l) {
  return a.axis && l.turn && l.mine ? *(const uint64_t*)(a.axis + l.u * 8) : 0;
}
template <bool PAIRS>
__device__ __forceinline__ void angles(const FormAppendArgs& a, const Lane<PAIRS>& l, const Where& w, uint64_t axis,
                                       Angles& v) {
  const int half = a.rot / 2;
  auto row = [&](int ax) __attribute__((always_inline)) {
    const int pos = ax == 0 ? w.pos[0] : (ax == 1 ? w.pos[1] : (ax == 2 ? w.pos[2] : w.pos[3]));
    return a.rope + (int64_t)pos * a.rot + l.u * 8;
  };
  if (axis == (axis & 0xff) * 0x0101010101010101ull && (int)(axis & 0xff) < a.axes) {  // one axis for all of them
    const float* at = row((int)(axis & 0xff));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t cv = *(const f32x4_t*)(at + 4 * i), sv = *(const f32x4_t*)(at + half + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v.c[4 * i + j] = cv[j];
        v.s[4 * i + j] = sv[j];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ax = (int)(axis >> (8 * i)) & 0xff;
      v.c[i] = 1.f;
      v.s[i] = 0.f;
      if (ax < a.axes) {
        const float* at = row(ax) + i;
        v.c[i] = at[0];
        v.s[i] = at[half];
      }
    }
  }
}
template <bool PAIRS>
__device__ __forceinline__ void turn(const Angles& v, float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = PAIRS ? 2 * i : i, ib = PAIRS ? 2 * i + 1 : 8 + i;
    const float p = x[ia], r = x[ib];
    x[ia] = fmaf(p, v.c[i], -(r * v.s[i]));
    x[ib] = fmaf(r, v.c[i], p * v.s[i]);
  }
}

// Four values over a scale as codes, rounded to nearest, ties to even;
// infinities become NaN.
typedef short s16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t codes4(const float* x, float scale) {
  s16x2_t w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], scale, false);
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], scale, true));
}

// The byte of the least scale for rows whose largest finite element is A.
__device__ __forceinline__ int need_byte(float A) {
  const uint32_t w = __float_as_uint(A);
  const int e = (int)(w >> 23) - 8 + ((w & 0x7fffffu) > 0x600000u ? 1 : 0);  // (448 = 1.75 * 2^8)
  return e < 1 ? 1 : e;
}

// What a workgroup knows of its window: kNear tokens before it, its own, and
// kNear behind.
constexpr int kXcds = 8;
constexpr int kNear = 15;  // tokens of a block stand no further apart
constexpr int kHeads = 2;  // of a workgroup, at most
template <int SPAN>
struct Window {
  int slot[SPAN + 2 * kNear];            // -1: padding
  float top[kHeads][SPAN + 2 * kNear];  // the row's largest finite magnitude
};

// Heads h0 .. h1 - 1 of the keys or values of the window from token t0 on.  A
// group of LPR lanes has the token of its number, and one beside the window whose
// block is also in it.
template <class T, int LPR, bool PAIRS, bool KEYS>
__device__ __forceinline__ void write_blocks(const FormAppendArgs& a, int t0, int h0, int h1,
                                             Window<kThreads / LPR>& w) {
  constexpr int SPAN = kThreads / LPR;
  const int tid = threadIdx.x, group = tid / LPR, lane = tid & 63;
  Lane<PAIRS> l(a, tid % LPR);
  if (!KEYS) {  // (values: whole neighbouring chunks)
    l.c0 = 2 * l.u;
    l.c1 = l.c0 + 1;
  }
  const bool turned = KEYS && l.turn && l.mine;
  struct Raw {
    u32x4_t w0, w1;
  };
  auto load = [&](int t, int h, bool on) __attribute__((always_inline)) {
    Raw r = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    if (on && l.mine) {
      const uint16_t* at = KEYS ? a.k + t * a.k_token + h * a.k_head : a.v + t * a.v_token + h * a.v_head;
      r.w0 = *(const u32x4_t*)(at + l.c0 * 8);
      r.w1 = *(const u32x4_t*)(at + l.c1 * 8);
    }
    return r;
  };
  // a row, and its largest finite magnitude
  auto make = [&](const Raw& r, const Angles& v, bool on, float* x) __attribute__((always_inline)) {
    widen8<T>(r.w0, x);
    widen8<T>(r.w1, x + 8);
    if (KEYS && a.k_weight) norm<LPR>(a, l, a.k_weight, x);
    if (on && turned) turn<PAIRS>(v, x);
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));  // (which is not NaN)
    if (__any(top > kLargest)) {
      top = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]) <= kLargest ? fabsf(x[k]) : 0.f);
    }
    return join_lanes<LPR>(top, [](float p, float q) { return fmaxf(p, q); });
  };

  const int t = t0 + group;
  Where mine = {-1, {0, 0, 0, 0}, false};
  if (t < a.T) mine = where(a, t);
  const int slot = mine.slot;
  const bool on = mine.live;
  const uint64_t axis = KEYS ? axes_of(a, l) : 0;
  Raw raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) raw[i] = load(t, h0 + i, t < a.T && h0 + i < h1);
  for (int i = tid; i < SPAN + 2 * kNear; i += kThreads) {
    const int64_t n = (int64_t)t0 - kNear + i;
    Where other = {-1, {0, 0, 0, 0}, false};
    if (n >= 0 && n < a.T) other = where(a, (int)n);
    w.slot[i] = other.live ? other.slot : -1;
  }
  Angles v;
  if (on && turned) angles(a, l, mine, axis, v);
  const int at = kNear + group, block = slot >> 4;
  const int page = on ? slot >> a.page_shift : 0, off = on ? slot & ((1 << a.page_shift) - 1) : 0;
  uint8_t* const scales = KEYS ? a.ks + page * a.ks_page + (off >> 4) : a.vs + page * a.vs_page + (off >> 4);
  uint8_t* const codes = KEYS ? a.k8 + page * a.kc_page + (off & ~15) * a.kc_slot
                              : a.v8 + page * a.vc_page + (off & ~15) * a.vc_slot;
  const int64_t head = KEYS ? a.kc_head : a.vc_head, step = KEYS ? a.kc_slot : a.vc_slot;
  const int64_t shead = KEYS ? a.ks_head : a.vs_head;
  int old[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) old[i] = on && h0 + i < h1 ? scales[(h0 + i) * shead] : 1;
  __syncthreads();
  // places of the block that the call writes, and whether this token is the first of them
  uint32_t held = 0, same = 0;  // bit c: the c-th of the places that this lane looks at is of the same block
  uint32_t before = 0;
#pragma unroll
  for (int c = 0; c < (2 * kNear + LPR) / LPR; ++c) {
    const int j = c * LPR + l.u, other = w.slot[min(group + j, SPAN + 2 * kNear - 1)];
    if (on && j <= 2 * kNear && other >> 4 == block) {
      held |= 1u << (other & 15);
      same |= 1u << c;
      before |= j < kNear;
    }
  }
  held = join_lanes<LPR>(held, [](uint32_t p, uint32_t q) { return p | q; });
  before = join_lanes<LPR>(before, [](uint32_t p, uint32_t q) { return p | q; });
  // rows beside the window
#pragma unroll 1
  for (int i = group; i < (2 * kNear + SPAN - 1) / SPAN * SPAN; i += SPAN) {
    const bool left = i < kNear;
    const int n = left ? i : SPAN + i, other = i < 2 * kNear ? w.slot[n] : -1;
    uint32_t need = 0;
#pragma unroll
    for (int c = 0; c < (kNear + LPR - 1) / LPR; ++c) {
      const int j = 1 + c * LPR + l.u, k = left ? n + j : n - j;
      if (j <= kNear && k >= kNear && k < kNear + SPAN && other >= 0) need |= w.slot[k] >> 4 == other >> 4;
    }
    need = join_lanes<LPR>(need, [](uint32_t p, uint32_t q) { return p | q; });
    Raw r[kHeads];
    Angles u;
    if (need) {
#pragma unroll
      for (int k = 0; k < kHeads; ++k) r[k] = load(t0 - kNear + n, h0 + k, h0 + k < h1);
      if (turned) angles(a, l, where(a, t0 - kNear + n), axis, u);
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        float y[16];
        const float top = make(r[k], u, true, y);
        if (l.u == 0) w.top[k][n] = top;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i;
    if (h >= h1) break;
    float x[16];
    float top = make(raw[i], v, on, x);
    if (l.u == 0) w.top[i][at] = top;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < (2 * kNear + LPR) / LPR; ++c) {
      const float other = w.top[i][min(group + c * LPR + l.u, SPAN + 2 * kNear - 1)];
      if ((same >> c) & 1) top = fmaxf(top, other);
    }
    top = join_lanes<LPR>(top, [](float p, float q) { return fmaxf(p, q); });
    // (another workgroup may have written the scale of a block that it shares: the larger of the two is the same)
    const bool begun = held & 1;
    const int was = begun ? 1 : (old[i] < 1 ? 1 : (old[i] > 254 ? 254 : old[i])), byte = max(need_byte(top), was);
    // older codes of a block whose scale grew, by the whole wavefront of the block's first token
    uint64_t grown = __ballot(on && !before && !begun && byte > was && l.u == 0);
    while (grown) {
      const int from = __builtin_ctzll(grown);
      grown &= grown - 1;
      const uint32_t kept = (uint32_t)__builtin_amdgcn_readlane((int)held, from);
      const float f = __builtin_ldexpf(1.f, __builtin_amdgcn_readlane(was - byte, from));
      const uint64_t base = (uint64_t)(codes + h * head);
      uint8_t* const to = (uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)base, from) |
                                     (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(base >> 32), from) << 32);
      for (int k = lane / LPR; k < 16; k += 64 / LPR) {
        if (((kept >> k) & 1) || !l.mine) continue;
        u32x4_t* const place = (u32x4_t*)(to + k * step + l.u * 16);
        u32x4_t c = *place;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q], false);
          const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q], true);
          const float y[4] = {lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f};
          c[q] = codes4(y, 1.f);
        }
        *place = c;
      }
    }
    if (on && l.mine) {
      const float f = block_scale((uint32_t)byte);
      uint8_t* const to = codes + h * head + (slot & 15) * step;
      *(u32x2_t*)(to + l.c0 * 8) = u32x2_t{codes4(x, f), codes4(x + 4, f)};
      *(u32x2_t*)(to + l.c1 * 8) = u32x2_t{codes4(x + 8, f), codes4(x + 12, f)};
    }
    if (on && !before && l.u == 0) scales[h * shead] = (uint8_t)byte;
  }
}

// Rows of queries, and with a 16-bit cache of keys and values.
template <class T, int LPR, bool PAIRS, bool F8>
__device__ __forceinline__ void write_row(const FormAppendArgs& a, int64_t row) {
  const int heads = F8 ? a.Hq : a.Hq + 2 * a.Hkv;
  if (row >= (int64_t)a.T * heads) return;  // (whole rows: the exchanges below stay inside a row)
  const Lane<PAIRS> l(a, threadIdx.x % LPR);
  const int t = (int)(row / heads), h = (int)(row - (int64_t)t * heads);
  const uint64_t axis = axes_of(a, l);
  const Where w = where(a, t);
  const int slot = w.slot;
  const bool live = w.live;
  const int off = slot & ((1 << a.page_shift) - 1), page = slot >> a.page_shift;
  const uint16_t* src;
  uint16_t* dst;
  if (h < a.Hq) {
    src = a.q + t * a.q_token + h * a.q_head;
    dst = a.out + t * a.o_token + h * a.o_head;
    if (!live) {
      if (l.mine) {
        *(u32x4_t*)(dst + l.c0 * 8) = u32x4_t{0u, 0u, 0u, 0u};
        *(u32x4_t*)(dst + l.c1 * 8) = u32x4_t{0u, 0u, 0u, 0u};
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
      if (l.mine) {
        const u32x4_t w0 = *(const u32x4_t*)(src + l.c0 * 8), w1 = *(const u32x4_t*)(src + l.c1 * 8);
        *(u32x4_t*)(dst + l.c0 * 8) = w0;
        *(u32x4_t*)(dst + l.c1 * 8) = w1;
      }
      return;
    }
  }
  u32x4_t w0 = {0u, 0u, 0u, 0u}, w1 = w0;
  if (l.mine) {
    w0 = *(const u32x4_t*)(src + l.c0 * 8);
    w1 = *(const u32x4_t*)(src + l.c1 * 8);
  }
  float x[16];
  widen8<T>(w0, x);
  widen8<T>(w1, x + 8);
  const float* weight = h < a.Hq ? a.q_weight : a.k_weight;
  if (weight) norm<LPR>(a, l, weight, x);
  if (l.turn && l.mine) {
    Angles v;
    angles(a, l, w, axis, v);
    turn<PAIRS>(v, x);
  }
  if (l.mine) {
    *(u32x4_t*)(dst + l.c0 * 8) = narrow8<T>(x);
    *(u32x4_t*)(dst + l.c1 * 8) = narrow8<T>(x + 8);
  }
}

// LPR: lanes per row, the power of two from D / 16 up.
template <class T, int LPR, bool PAIRS, bool F8>
__global__ __launch_bounds__(kThreads, F8 ? 4 : 8) void append_form_kernel(FormAppendArgs a) {
  constexpr int kRows = kThreads / LPR;
  int64_t group = blockIdx.x;
  if constexpr (F8) {
    __shared__ Window<kRows> w;
    if (group < a.writers) {  // (they take longest, and come first)
      // Keys and values of `some` heads.  Workgroups go to the 8 XCDs in turn: all of a window's go to one, so that its
      // angles stay in one L2 and each has as many of the keys, which take longer than values.
      const int parts = (a.Hkv + a.some - 1) / a.some, i = (int)(group / kXcds), part = i % (2 * parts);
      const int64_t t0 = ((int64_t)(i / (2 * parts)) * kXcds + (int)(group % kXcds)) * kRows;
      const int h0 = part % parts * a.some, h1 = min(h0 + a.some, a.Hkv);
      if (t0 >= a.T) return;
      if (part < parts)
        write_blocks<T, LPR, PAIRS, true>(a, (int)t0, h0, h1, w);
      else if (a.v)
        write_blocks<T, LPR, PAIRS, false>(a, (int)t0, h0, h1, w);
      return;
    }
    group -= a.writers;
  }
  write_row<T, LPR, PAIRS, F8>(a, group * kRows + threadIdx.x / LPR);
}

// Queries of more workgroups than this have a launch of their own.  Measured, the append alone (bf16), with the writers
// / apart: 32 + 8 heads of 128 2,047 workgroups 15.9 / 20.3 us, 4,095 26.7 / 32.6, 8,191 54.3 / 57.7, 16,001 101.8 /
// 97.1; 28 + 4 heads by 3 axes 3,583 22.3 / 25.9, 5,250 36.4 / 37.9, 7,167 48.4 / 44.9, 14,000 92.2 / 76.9; 16 + 8 heads
// of 256 8,191 77.1 / 81.9.  (So the two meet between 5,500 and 12,000 or later by shape, and from here to there apart
// costs up to 20%.)
constexpr int64_t kApart = 4096;
// Workgroups for each compute unit from which two heads share one.  Measured, one head / two, by windows times heads: 8
// heads of 128 512 11.7 / 12.6 us, 752 16.0 / 14.1, 1,024 19.0 / 16.3, 4,008 71.4 / 55.8; 4 heads by 3 axes 376 12.4 /
// 12.9, 512 14.4 / 13.9, 1,024 22.5 / 20.6; 8 heads of 256 504 14.5 / 15.1, 1,024 22.5 / 19.9; 16 heads of 64 512 11.6 /
// 12.7, 752 15.4 / 13.9.  (They meet between 450 and 700.)
constexpr int64_t kPerCu = 4;

template <class T, int LPR>
void launch_lpr(FormAppendArgs a, bool eight, bool interleaved, hipStream_t stream) {
  if (eight) {
    // Two heads share the look at the window where that leaves each compute unit kPerCu workgroups.
    const int64_t windows = (a.T + kThreads / LPR - 1) / (kThreads / LPR);
    a.some = windows * a.Hkv >= kPerCu * kComputeUnits ? kHeads : 1;
    a.writers = (int)((windows + kXcds - 1) / kXcds * kXcds * 2 * ((a.Hkv + a.some - 1) / a.some));
  }
  // Writers hold twice the registers of rows, so the queries of a large call take a launch of their own.
  const int64_t rows = (int64_t)a.T * (eight ? a.Hq : a.Hq + 2 * a.Hkv), per = kThreads / LPR;
  const int64_t groups = (rows + per - 1) / per;
  const bool apart = eight && groups > kApart;
  if (eight) {
    const dim3 grid((unsigned)(a.writers + (apart ? 0 : groups)));
    if (interleaved)
      append_form_kernel<T, LPR, true, true><<<grid, kThreads, 0, stream>>>(a);
    else
      append_form_kernel<T, LPR, false, true><<<grid, kThreads, 0, stream>>>(a);
    if (!apart) return;
    a.Hkv = 0;
  }
  const dim3 grid((unsigned)groups);
  if (interleaved)
    append_form_kernel<T, LPR, true, false><<<grid, kThreads, 0, stream>>>(a);
  else
    append_form_kernel<T, LPR, false, false><<<grid, kThreads, 0, stream>>>(a);
}

template <class T>
void launch_type(const FormAppendArgs& a, bool eight, bool interleaved, hipStream_t stream) {
  if (a.D <= 32)
    launch_lpr<T, 2>(a, eight, interleaved, stream);
  else if (a.D <= 64)
    launch_lpr<T, 4>(a, eight, interleaved, stream);
  else if (a.D <= 128)
    launch_lpr<T, 8>(a, eight, interleaved, stream);
  else
    launch_lpr<T, 16>(a, eight, interleaved, stream);
}

// 16 codes of a row and head as 16-bit values.
template <class T>
__device__ __forceinline__ void read16(const uint8_t* src, const uint8_t* scale, bool live, uint16_t* dst) {
  u32x4_t c = {0u, 0u, 0u, 0u};
  float f = 0.f;
  if (live) {
    c = *(const u32x4_t*)src;
    f = block_scale(*scale);
  }
  u32x4_t o[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i / 2][i % 2 * 2] = code_pair<T, false>(c[i], f);
    o[i / 2][i % 2 * 2 + 1] = code_pair<T, true>(c[i], f);
  }
  *(u32x4_t*)dst = o[0];
  *(u32x4_t*)(dst + 8) = o[1];
}

template <class T>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
  const int per = a.D / 16;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, row = i / per;
  const int u = (int)(i - row * per);
  if (row >= (int64_t)a.n * a.heads) return;
  const int r = (int)(row / a.heads), h = (int)(row - (int64_t)r * a.heads);
  int slot = a.slots ? a.slots[r] : r;
  const bool live = slot >= 0 && slot < a.num_slots;
  if (!live) slot = 0;
  const int64_t page = slot >> a.page_shift;
  const int off = slot & ((1 << a.page_shift) - 1);
  if (a.ko)
    read16<T>(a.k + page * a.k_page + off * a.k_slot + h * a.k_head + u * 16,
              a.ks + page * a.ks_page + h * a.ks_head + (off >> 4), live, a.ko + r * a.ko_row + h * a.ko_head + u * 16);
  if (a.vo)
    read16<T>(a.v + page * a.v_page + off * a.v_slot + h * a.v_head + u * 16,
              a.vs + page * a.vs_page + h * a.vs_head + (off >> 4), live, a.vo + r * a.vo_row + h * a.vo_head + u * 16);
}

}  // namespace

hipError_t launch_append_form(const FormAppendArgs& a, int dt, bool eight, bool interleaved, hipStream_t stream) {
  if (dt == 1)
    launch_type<BF16>(a, eight, interleaved, stream);
  else
    launch_type<F16>(a, eight, interleaved, stream);
  return hipGetLastError();
}

hipError_t launch_read(const ReadArgs& a, int dt, hipStream_t stream) {
  const int64_t threads = (int64_t)a.n * a.heads * (a.D / 16);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  if (dt == 1)
    read_kernel<BF16><<<grid, kThreads, 0, stream>>>(a);
  else
    read_kernel<F16><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace kmkv

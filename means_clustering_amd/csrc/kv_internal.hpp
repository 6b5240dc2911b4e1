// Internal declarations of the paged key/value cache library (gfx950 /
// MI355X only).  Nothing here is part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kmkv {

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

// 16-bit element types: two elements packed in 32 bits, widened or rounded
// (to nearest, ties to even), what an element's exponent looks like when it is
// infinite or NaN, and the power of two that softmax terms are held times, so
// that those far below the largest (which is 1 before) keep their bits: fp16
// has full ones down to 2^-14 and none below 2^-25.
struct BF16 {
  static constexpr uint32_t kExp = 0x7f80u;
  static constexpr float kTerm = 0.f;
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
  }
};
struct F16 {
  static constexpr uint32_t kExp = 0x7c00u;
  static constexpr float kTerm = 14.f;
  static __device__ __forceinline__ float lo(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xffffu));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, (f16x2_t){(_Float16)a, (_Float16)b});
  }
};

// Inclusive sums over the wavefront (row shifts, then row broadcasts).
template <int CTRL, int ROWS, class V>
__device__ __forceinline__ V dpp_(V v) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
  } else {
    const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
    return __builtin_bit_cast(V, u32x2_t{(unsigned)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xf, false),
                                         (unsigned)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xf, false)});
  }
}
template <class V>
__device__ __forceinline__ V wave_scan(V v) {
  v += dpp_<0x111, 0xf>(v);
  v += dpp_<0x112, 0xf>(v);
  v += dpp_<0x114, 0xf>(v);
  v += dpp_<0x118, 0xf>(v);
  v += dpp_<0x142, 0xa>(v);
  v += dpp_<0x143, 0xc>(v);
  return v;
}

// ------------------------------------------------------------------ tables ----

struct TablesArgs {
  const int32_t *ctx, *fresh, *offset;
  int32_t R;
  int32_t page_shift;
  int32_t* table;
  int64_t table_stride;
  int32_t width;
  const int32_t* free_pages;
  int32_t num_free;
  int32_t T;
  int32_t *seq_lens, *query_start, *page_start, *positions, *slots;
};
hipError_t launch_tables(const TablesArgs& a, hipStream_t stream);

// ------------------------------------------------------------------ append ----

struct AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // elements
  uint16_t* out;
  int64_t o_token, o_head;
  uint16_t *kc, *vc;
  int64_t kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;
  const float *q_weight, *k_weight, *rope;
  const int32_t *positions, *slots;
  int32_t T, Hq, Hkv, D, rot;
  int32_t max_pos, num_slots, page_shift;
  float eps;
};
hipError_t launch_append(const AppendArgs& a, int dt, bool interleaved, hipStream_t stream);

// ------------------------------------------------------------------ attend ----

struct AttendArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_token, q_head, o_token, o_head;  // elements
  const uint8_t *k, *v;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // bytes
  int32_t pages, page_shift;
  const int32_t* table;
  int64_t table_stride;
  int32_t width;
  const int32_t *query_start, *seq_lens;
  const float* lw;
  int64_t lw_page, lw_head;  // elements
  int32_t R, T, Hq, Hkv, G, D;
  int32_t window;    // 0: none
  float scale;       // without weights times log2(e)
  // The launch handles the requests with more than lo_rows and at most
  // hi_rows rows (new tokens x G).
  int64_t lo_rows, hi_rows;
  int32_t pieces;     // decode: workgroups
  int64_t* per_head;  // decode: units of all requests, for one head (written)
  int32_t target;     // chunk: items per cache head that the keys are divided into
  int32_t min_units;  // chunk: least key units of an item
  int32_t max_items;  // chunk: items per cache head, at most
  int32_t parts;      // chunk: parts that the workspace holds
  // Results of shared rows: o relative to its m, m and l.  Decode: rows
  // [2 * pieces][BM], two for a workgroup (of its first request, and of its
  // last if that is another); chunk: rows [parts][Hkv][BM].
  float* part_o;
  f32x2_t* part_ml;
  // [T] for the join.  Decode: (position of the request's first unit, its
  // units, token in the request, upper half of the position * 2); chunk:
  // (first part, splits, token in the request, 1).
  int4* info;
};

constexpr int kDecodeUnit = 128;  // keys per step of a decode workgroup: 32 for each of its 4 wavefronts
// Decode workgroups that a compute unit holds (by their registers).
constexpr int decode_per_cu(int dpad, int bm) {
  return dpad == 64 ? (bm == 16 ? 3 : 2) : (dpad == 128 && bm == 16 ? 2 : 1);
}
constexpr int kComputeUnits = 256;  // of an MI355X; with fewer the pieces take turns
constexpr int kChunkRows = 128;   // rows of a chunk workgroup: 32 for each of its 4 wavefronts
constexpr int chunk_unit(int dpad) { return dpad > 128 ? 32 : 64; }  // keys per step of a chunk workgroup
inline int dim_pad(int64_t D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

// One decode launch (BM = 16 or 32 rows), one chunk launch, and the join of
// the parts of rows whose keys were divided.
hipError_t launch_decode(const AttendArgs& a, int dt, int bm, hipStream_t stream);
hipError_t launch_chunk(const AttendArgs& a, int dt, hipStream_t stream);
struct JoinArgs {
  const float *o0, *o1;        // parts of the decode and of the chunk launch
  const f32x2_t *ml0, *ml1;
  int32_t bm0, pieces, parts1;
  const int64_t* per_head;
  const int4* info;
  uint16_t* out;
  float* lse;
  int64_t o_token, o_head;
  const int32_t* query_start;
  int32_t R, T, Hq, Hkv, G, D;
  bool weighted;
};
hipError_t launch_join(const JoinArgs& a, int dt, hipStream_t stream);

}  // namespace kmkv

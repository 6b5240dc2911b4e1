// C ABI of the paged key/value cache: argument checks, and how the attention
// divides its work.
#include <algorithm>
#include <limits>
#include <string>

#include "../../include/kmeans_cache.h"
#include "kv_internal.hpp"

using namespace kmkv;

namespace {

thread_local std::string g_error;

km_status fail(km_status s, const char* msg) noexcept {
  try {
    g_error = msg;
  } catch (...) {
  }
  return s;
}
km_status invalid(const char* msg) noexcept { return fail(KM_ERR_INVALID_VALUE, msg); }
km_status launched(hipError_t e) noexcept {
  return e == hipSuccess ? KM_OK : fail(KM_ERR_HIP, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
constexpr int64_t kMaxI = ((int64_t)1 << 31) - 1, kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxRoom = (int64_t)1 << 30;  // slots of a row of the block table
// A launch has fewer than 2^32 threads: workgroups of 256, which take at least
// 16 rows of the append, or an item or a token of the attention.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1, kMaxRows = 16 * kMaxGroups;

int shift_of(int64_t page_size) {
  int s = 0;
  while (((int64_t)1 << s) < page_size) ++s;
  return s;
}

bool page_size_ok(int64_t p) { return p >= 16 && p <= (1 << 20) && (p & (p - 1)) == 0; }

// Token and head strides of 16-byte aligned rows.
bool rows_ok(const void* p, int64_t token, int64_t head) {
  return p && aligned(p, 16) && token % 8 == 0 && head % 8 == 0 && token >= 0 && head >= 0 && token < kMaxStride &&
         head < kMaxStride;
}

const char* cache_error(const km_kv_cache* c, bool need_v) {
  if (!c) return "the cache is NULL";
  if (c->heads < 1 || c->heads > (1 << 16)) return "cache heads must be 1 to 65536";
  if (c->dim < 16 || c->dim > 256 || c->dim % 16) return "cache dim must be a multiple of 16 up to 256";
  if (!page_size_ok(c->page_size)) return "page_size must be a power of two from 16 to 2^20";
  if (c->pages < 1 || c->pages > kMaxI / c->page_size)
    return "pages must be at least 1 and pages * page_size below 2^31";
  if (!rows_ok(c->k, c->k_page, c->k_slot) || !rows_ok(c->k, c->k_head, 0))
    return "cache keys must be 16-byte aligned with strides that are multiples of 8";
  if (need_v && (!rows_ok(c->v, c->v_page, c->v_slot) || !rows_ok(c->v, c->v_head, 0)))
    return "cache values must be 16-byte aligned with strides that are multiples of 8";
  return nullptr;
}

// How an attention call is divided into launches, and its workspace.
struct Plan {
  bool decode = false, chunk = false;
  int bm = 16;                // decode rows
  int64_t pieces = 0;         // decode workgroups
  int64_t target = 0;         // chunk: items wanted per cache head
  int64_t tiles = 0;          // ... tiles, at most
  int64_t parts[2] = {0, 0};  // rows of parts: decode, chunk
  size_t head_at = 0, info_at = 256, o_at[2] = {0, 0}, ml_at[2] = {0, 0}, bytes = 0;
};

// Chunk items in all: as many as the GPU holds at once, two for a compute
// unit.  (Measured: 509 tokens over 30,000 slots 294 us; 360, 316 and 350 us
// with 768, 1,024 and 2,048 items.  Items have at least 4 tiles: of 1 or 8, a
// chunk of 65 tokens takes 25 us instead of 24.)
constexpr int64_t kChunkGroups = 512;
constexpr int kChunkMinUnits = 4;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

Plan make_plan(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t R, int64_t max_new) {
  Plan p;
  const int64_t G = Hq / Hkv, most = std::min(max_new, T), rows = most * G;
  // Requests of up to 16 rows take the decode launch, of more rows the chunk
  // launch; up to 32 rows a wider decode launch serves all.  (Measured, bf16,
  // 8 heads of 128: 63 requests of 20 rows 164 us in the decode launch, 228 in
  // the chunk launch, 32 rows over a quarter of the keys 57 against 68; wider
  // ones would leave a compute unit one wavefront a SIMD.)
  p.bm = rows <= 16 ? 16 : (rows <= 32 ? 32 : 16);
  p.chunk = rows > 32;
  p.decode = !p.chunk || (R > 1 && G <= 16);
  const int dp = dim_pad(D);
  if (p.decode) {
    p.pieces = (int64_t)kComputeUnits * decode_per_cu(dp, p.bm);
    p.parts[0] = 2 * p.pieces;
  }
  if (p.chunk) {
    p.target = std::max<int64_t>(1, kChunkGroups / Hkv);
    p.tiles = std::min(R * ((rows + kChunkRows - 1) / kChunkRows), T * G / kChunkRows + R);
    p.parts[1] = std::min(2 * p.target, p.target + p.tiles);
  }
  size_t at = p.info_at + up256((size_t)T * sizeof(int4));
  for (int i = 0; i < 2; ++i) {
    const size_t n = (size_t)p.parts[i] * (size_t)(i ? Hkv * kChunkRows : p.bm);
    p.o_at[i] = at;
    at += up256(n * (size_t)dp * sizeof(float));
    p.ml_at[i] = at;
    at += up256(n * sizeof(f32x2_t));
  }
  p.bytes = at;
  return p;
}

const char* attend_error(const km_kv_cache* c, int64_t T, int64_t Hq, int64_t R, int64_t max_new) {
  if (const char* e = cache_error(c, true)) return e;
  if (T < 0 || T > kMaxGroups || R < 0 || R > kMaxGroups) return "T and R must be 0 to 2^24 - 1";
  // (the join has a workgroup row for every 4 query heads or more, and a launch 65,535 of them)
  if (Hq < 1 || Hq % c->heads || Hq > (1 << 17)) return "q_heads must be a multiple of the cache's heads up to 2^17";
  if (T * Hq > kMaxI) return "T * q_heads must be below 2^31";
  if (max_new < 0 || max_new > kMaxI) return "max_new must be 0 to 2^31 - 1";
  return nullptr;
}

}  // namespace

extern "C" km_status kmeans_kv_tables(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* pos_offset,
                                      int64_t R, int64_t page_size, int32_t* block_table, int64_t width,
                                      int64_t table_stride, const int32_t* free_pages, int64_t num_free, int64_t T,
                                      int32_t* seq_lens, int32_t* query_start, int32_t* page_start,
                                      int32_t* positions, int32_t* slots, void* stream) {
  if (R < 0 || R > kMaxGroups || T < 0 || T > kMaxI)
    return invalid("R must be 0 to 2^24 - 1 and T 0 to 2^31 - 1");
  if (!page_size_ok(page_size)) return invalid("page_size must be a power of two from 16 to 2^20");
  if (width < 0 || width > kMaxI / page_size || table_stride < width || table_stride >= kMaxStride)
    return invalid("width must be at least 0, width * page_size below 2^31 and table_stride at least width");
  if (num_free < 0 || num_free > kMaxI) return invalid("num_free must be 0 to 2^31 - 1");
  if (!query_start || !page_start) return invalid("query_start and page_start must not be NULL");
  if (R > 0 && (!ctx_lens || !new_lens || !seq_lens || (width > 0 && !block_table)))
    return invalid("ctx_lens, new_lens, seq_lens and block_table must not be NULL");
  if (num_free > 0 && !free_pages) return invalid("free_pages must not be NULL");
  if (T > 0 && (!positions || !slots)) return invalid("positions and slots must not be NULL");
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)pos_offset,
                        (const void*)block_table, (const void*)free_pages, (const void*)seq_lens,
                        (const void*)query_start, (const void*)page_start, (const void*)positions,
                        (const void*)slots})
    if (!aligned(p, 4)) return invalid("pointers must be 4-byte aligned");
  // the workgroups read the lengths for themselves, at different times
  // (arrays of no elements may have any address)
  const void *token_out[2] = {T > 0 ? positions : nullptr, T > 0 ? slots : nullptr};
  for (const void* out : {(const void*)seq_lens, (const void*)query_start, (const void*)page_start, token_out[0],
                          token_out[1]})
    for (const void* in : {(const void*)ctx_lens, (const void*)new_lens, (const void*)pos_offset,
                           (const void*)(num_free > 0 ? free_pages : nullptr)})
      if (R > 0 && out && out == in) return invalid("an output must not be an input");
  TablesArgs a;
  a.ctx = ctx_lens;
  a.fresh = new_lens;
  a.offset = pos_offset;
  a.R = (int32_t)R;
  a.page_shift = shift_of(page_size);
  a.table = block_table;
  a.table_stride = table_stride;
  a.width = (int32_t)width;
  a.free_pages = free_pages;
  a.num_free = (int32_t)num_free;
  a.T = (int32_t)T;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.page_start = page_start;
  a.positions = positions;
  a.slots = slots;
  return launched(launch_tables(a, (hipStream_t)stream));
}

extern "C" km_status kmeans_kv_append(const km_kv_cache* cache, km_dtype dt, int64_t T, const void* q, int64_t q_heads,
                                      int64_t q_token, int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                                      const void* v, int64_t v_token, int64_t v_head, const float* q_weight,
                                      const float* k_weight, float eps, const int32_t* positions, const float* rope,
                                      int64_t max_pos, int64_t rot, int interleaved, const int32_t* slots, void* q_out,
                                      int64_t o_token, int64_t o_head, void* stream) {
  if (const char* e = cache_error(cache, v != nullptr)) return invalid(e);
  if (dt == KM_F32) return fail(KM_ERR_UNSUPPORTED, "the cache holds KM_BF16 or KM_F16");
  if (dt != KM_BF16 && dt != KM_F16) return invalid("dtype must be KM_BF16 or KM_F16");
  if (q_heads < 0 || q_heads > (1 << 20)) return invalid("q_heads must be 0 to 2^20");
  if (T < 0 || T > kMaxI) return invalid("T must be 0 to 2^31 - 1");
  if (T * (q_heads + 2 * cache->heads) > kMaxRows)
    return fail(KM_ERR_UNSUPPORTED, "T * (q_heads + 2 * heads) must be at most 2^28 - 16");
  if (!(eps >= 0.f)) return invalid("eps must not be negative");
  if (rot < 0 || rot > cache->dim || rot % 16) return invalid("rot must be a multiple of 16 up to the cache's dim");
  if (rot > 0 && (!rope || !positions || max_pos < 1 || max_pos > kMaxI))
    return invalid("a rotation needs rope, positions and max_pos from 1 to 2^31 - 1");
  if (rot == 0 && (rope || positions)) return invalid("rope and positions must be NULL where rot is 0");
  if (!aligned(rope, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return invalid("rope, q_weight and k_weight must be 16-byte aligned");
  if (!aligned(positions, 4) || !aligned(slots, 4)) return invalid("positions and slots must be 4-byte aligned");
  if (T == 0) return KM_OK;
  if (q_heads > 0 && (!rows_ok(q, q_token, q_head) || !rows_ok(q_out, o_token, o_head)))
    return invalid("q and q_out must be 16-byte aligned with strides that are multiples of 8");
  if (!rows_ok(k, k_token, k_head)) return invalid("k must be 16-byte aligned with strides that are multiples of 8");
  if (v && !rows_ok(v, v_token, v_head))
    return invalid("v must be 16-byte aligned with strides that are multiples of 8");
  if (q_heads > 0 && q == q_out && (q_token != o_token || q_head != o_head))
    return invalid("q_out may be q itself only with the same strides");
  AppendArgs a;
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q_token = q_token;
  a.q_head = q_head;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.out = (uint16_t*)q_out;
  a.o_token = o_token;
  a.o_head = o_head;
  a.kc = (uint16_t*)cache->k;
  a.vc = (uint16_t*)cache->v;
  a.kc_page = cache->k_page;
  a.kc_slot = cache->k_slot;
  a.kc_head = cache->k_head;
  a.vc_page = cache->v_page;
  a.vc_slot = cache->v_slot;
  a.vc_head = cache->v_head;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.rope = rope;
  a.positions = positions;
  a.slots = slots;
  a.T = (int32_t)T;
  a.Hq = (int32_t)q_heads;
  a.Hkv = (int32_t)cache->heads;
  a.D = (int32_t)cache->dim;
  a.rot = (int32_t)rot;
  a.max_pos = rot > 0 ? (int32_t)max_pos : 1;
  a.num_slots = (int32_t)(cache->pages * cache->page_size);
  a.page_shift = shift_of(cache->page_size);
  a.eps = eps;
  return launched(launch_append(a, (int)dt, interleaved != 0, (hipStream_t)stream));
}

extern "C" size_t kmeans_kv_attend_workspace(const km_kv_cache* cache, int64_t T, int64_t q_heads, int64_t R,
                                             int64_t max_new) {
  if (attend_error(cache, T, q_heads, R, max_new)) return 0;
  return std::max<size_t>(256, make_plan(T, q_heads, cache->heads, cache->dim, R, max_new).bytes);
}

extern "C" km_status kmeans_kv_attend(const km_kv_cache* cache, km_dtype dt, const void* q, int64_t T, int64_t q_heads,
                                      int64_t q_token, int64_t q_head, const int32_t* block_table, int64_t R,
                                      int64_t width, int64_t table_stride, const int32_t* query_start,
                                      const int32_t* seq_lens, const float* log_weight, int64_t lw_page,
                                      int64_t lw_head, float scale, int64_t window, int64_t max_new, void* out,
                                      int64_t o_token, int64_t o_head, float* lse, void* ws, size_t ws_bytes,
                                      void* stream) {
  if (const char* e = attend_error(cache, T, q_heads, R, max_new)) return invalid(e);
  if (dt == KM_F32) return fail(KM_ERR_UNSUPPORTED, "the cache holds KM_BF16 or KM_F16");
  if (dt != KM_BF16 && dt != KM_F16) return invalid("dtype must be KM_BF16 or KM_F16");
  if (window < 0 || window > kMaxI) return invalid("window must be 0 (none) to 2^31 - 1");
  // (without weights the scores are in units of log 2)
  const float unit = log_weight ? scale : scale * 1.4426950408889634f;
  if (!(unit - unit == 0.f)) return invalid("scale must be finite, times log2(e) too");
  if (width < 0 || width > kMaxRoom / cache->page_size || table_stride < width || table_stride >= kMaxStride)
    return invalid("width must be at least 0, width * page_size at most 2^30 and table_stride at least width");
  if (T == 0 || R == 0 || max_new == 0) return KM_OK;
  if (!rows_ok(q, q_token, q_head) || !rows_ok(out, o_token, o_head))
    return invalid("q and out must be 16-byte aligned with strides that are multiples of 8");
  if (!query_start || !seq_lens || (width > 0 && !block_table))
    return invalid("query_start, seq_lens and block_table must not be NULL");
  if (!aligned(query_start, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(lse, 4))
    return invalid("query_start, seq_lens, block_table and lse must be 4-byte aligned");
  if (log_weight && (!aligned(log_weight, 16) || lw_page % 4 || lw_head % 4 || lw_page < 0 || lw_head < 0 ||
                     lw_page >= kMaxStride || lw_head >= kMaxStride))
    return invalid("log_weight must be 16-byte aligned with strides that are multiples of 4");
  const Plan p = make_plan(T, q_heads, cache->heads, cache->dim, R, max_new);
  if (R * cache->heads > kMaxGroups || (p.target + p.tiles) * cache->heads > kMaxGroups)
    return fail(KM_ERR_UNSUPPORTED, "too many requests, rows and heads for one launch");
  if (!ws || ws_bytes < p.bytes) return fail(KM_ERR_WORKSPACE, "the workspace is NULL or too small");
  if (!aligned(ws, 256)) return invalid("the workspace must be 256-byte aligned");
  AttendArgs a;
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.q_token = q_token;
  a.q_head = q_head;
  a.o_token = o_token;
  a.o_head = o_head;
  a.k = (const uint8_t*)cache->k;
  a.v = (const uint8_t*)cache->v;
  a.k_page = 2 * cache->k_page;
  a.k_slot = 2 * cache->k_slot;
  a.k_head = 2 * cache->k_head;
  a.v_page = 2 * cache->v_page;
  a.v_slot = 2 * cache->v_slot;
  a.v_head = 2 * cache->v_head;
  a.pages = (int32_t)cache->pages;
  a.page_shift = shift_of(cache->page_size);
  a.table = block_table;
  a.table_stride = table_stride;
  a.width = (int32_t)width;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.lw = log_weight;
  a.lw_page = lw_page;
  a.lw_head = lw_head;
  a.R = (int32_t)R;
  a.T = (int32_t)T;
  a.Hq = (int32_t)q_heads;
  a.Hkv = (int32_t)cache->heads;
  a.G = (int32_t)(q_heads / cache->heads);
  a.D = (int32_t)cache->dim;
  // A window of more than every position (at most 2^30) is none.  (Not one of the table row's room: a request that is
  // longer than its row has queries beyond it, from which the window hides slots of the row.)
  a.window = window >= kMaxRoom ? 0 : (int32_t)window;
  a.scale = unit;
  uint8_t* base = (uint8_t*)ws;
  a.per_head = (int64_t*)(base + p.head_at);
  a.info = (int4*)(base + p.info_at);
  // most keys that a tile can see, and whether any tile's keys can be divided
  const int64_t room = width * cache->page_size;
  const int64_t keys = std::max<int64_t>(1, a.window ? std::min<int64_t>(room, a.window + max_new + 256) : room);
  bool divided = false;
  if (p.decode) {
    const int64_t units = (keys + kDecodeUnit - 1) / kDecodeUnit;
    a.lo_rows = 0;
    a.hi_rows = p.bm;
    a.pieces = (int32_t)p.pieces;
    a.part_o = (float*)(base + p.o_at[0]);
    a.part_ml = (f32x2_t*)(base + p.ml_at[0]);
    divided = units > 1;
    const hipError_t e = launch_decode(a, (int)dt, p.bm, (hipStream_t)stream);
    if (e != hipSuccess) return launched(e);
  }
  if (p.chunk) {
    const int64_t unit = chunk_unit(dim_pad(cache->dim)), units = (keys + unit - 1) / unit;
    a.lo_rows = p.decode ? p.bm : 0;
    a.hi_rows = std::numeric_limits<int64_t>::max();
    a.target = (int32_t)p.target;
    a.min_units = kChunkMinUnits;
    const int64_t most = (units + a.min_units - 1) / a.min_units;
    a.max_items = (int32_t)std::min(p.target + p.tiles, p.tiles * most);
    a.parts = (int32_t)p.parts[1];
    a.part_o = (float*)(base + p.o_at[1]);
    a.part_ml = (f32x2_t*)(base + p.ml_at[1]);
    divided = divided || most > 1;
    const hipError_t e = launch_chunk(a, (int)dt, (hipStream_t)stream);
    if (e != hipSuccess) return launched(e);
  }
  if (!divided) return KM_OK;
  JoinArgs j;
  j.o0 = (const float*)((uint8_t*)ws + p.o_at[0]);
  j.o1 = (const float*)((uint8_t*)ws + p.o_at[1]);
  j.ml0 = (const f32x2_t*)((uint8_t*)ws + p.ml_at[0]);
  j.ml1 = (const f32x2_t*)((uint8_t*)ws + p.ml_at[1]);
  j.bm0 = p.bm;
  j.pieces = (int32_t)p.pieces;
  j.parts1 = (int32_t)p.parts[1];
  j.per_head = a.per_head;
  j.info = a.info;
  j.out = a.out;
  j.lse = lse;
  j.o_token = o_token;
  j.o_head = o_head;
  j.query_start = query_start;
  j.R = a.R;
  j.T = a.T;
  j.Hq = a.Hq;
  j.Hkv = a.Hkv;
  j.G = a.G;
  j.D = a.D;
  j.weighted = log_weight != nullptr;
  return launched(launch_join(j, (int)dt, (hipStream_t)stream));
}

extern "C" const char* kmeans_kv_last_error(void) { return g_error.c_str(); }

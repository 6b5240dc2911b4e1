// C ABI of the further forms of the paged key/value cache: argument checks.
#include <cmath>

#include "../../include/kmeans_cache_forms.h"
#include "kv_plan.hpp"

using namespace kmkv;

namespace {

// An 8-bit cache's rows are 16-byte aligned with strides of bytes.
bool codes_ok(const void* p, int64_t page, int64_t slot, int64_t head) {
  if (!p || !aligned(p, 16)) return false;
  for (int64_t s : {page, slot, head})
    if (s < 0 || s % 16 || s >= kMaxStride) return false;
  return true;
}

const char* codes_error(const km_kv_cache* c, const km_kv_scales* s, bool need_k, bool need_v) {
  if (!c) return "the cache is NULL";
  // (whatever is not needed stands for itself in the checks of the common limits)
  km_kv_cache common = *c;
  common.k = common.v = (void*)(uintptr_t)16;
  common.k_page = common.k_slot = common.k_head = common.v_page = common.v_slot = common.v_head = 16;
  if (const char* e = cache_error(&common, true)) return e;
  if ((need_k && !codes_ok(c->k, c->k_page, c->k_slot, c->k_head)) ||
      (need_v && !codes_ok(c->v, c->v_page, c->v_slot, c->v_head)))
    return "codes must be 16-byte aligned with strides that are multiples of 16";
  if ((need_k && !s->k) || (need_v && !s->v)) return "the scales are NULL";
  if (need_k && need_v && s->k == s->v) return "the scales of keys and values must be different arrays";
  const int64_t blocks = c->page_size / 16;
  for (int i = 0; i < 2; ++i) {
    const int64_t page = i ? s->v_page : s->k_page, head = i ? s->v_head : s->k_head;
    if (!(i ? need_v : need_k)) continue;
    if (head < blocks || head >= kMaxStride || page < (c->heads - 1) * head + blocks || page >= kMaxStride)
      return "the scales of heads and pages must not overlap, strides below 2^40";
  }
  return nullptr;
}

// Whether pages, slots and heads of codes lie apart: in the order of their strides each steps over all of the smaller
// ones.  (What the move of older codes reads nobody else writes then.)
bool apart(const km_kv_cache* c, int64_t page, int64_t slot, int64_t head) {
  struct {
    int64_t step, n;
  } d[3] = {{page, c->pages}, {slot, c->page_size}, {head, c->heads}};
  std::sort(d, d + 3, [](const auto& x, const auto& y) { return x.step < y.step; });
  int64_t span = c->dim;  // (no stride reaches kMaxStride)
  for (const auto& i : d) {
    if (i.n == 1) continue;
    if (i.step < span) return false;
    span = i.n - 1 > (kMaxStride - span) / i.step ? kMaxStride : span + (i.n - 1) * i.step;
  }
  return true;
}

km_status dtype_error(km_dtype dt) {
  if (dt == KM_F32) return fail(KM_ERR_UNSUPPORTED, "the type must be KM_BF16 or KM_F16");
  if (dt != KM_BF16 && dt != KM_F16) return invalid("dtype must be KM_BF16 or KM_F16");
  return KM_OK;
}

void take_cache(AttendArgs& a, const km_kv_cache* c, int bytes) {
  a.k = (const uint8_t*)c->k;
  a.v = (const uint8_t*)c->v;
  a.k_page = bytes * c->k_page;
  a.k_slot = bytes * c->k_slot;
  a.k_head = bytes * c->k_head;
  a.v_page = bytes * c->v_page;
  a.v_slot = bytes * c->v_slot;
  a.v_head = bytes * c->v_head;
  a.pages = (int32_t)c->pages;
  a.page_shift = shift_of(c->page_size);
  a.Hkv = (int32_t)c->heads;
  a.D = (int32_t)c->dim;
}

// attend_error, for either cache.
const char* form_error(const km_kv_cache* c, const km_kv_scales* s, int64_t T, int64_t Hq, int64_t R,
                       int64_t max_new) {
  if (!s) return attend_error(c, T, Hq, R, max_new);
  if (const char* e = codes_error(c, s, true, true)) return e;
  km_kv_cache common = *c;
  common.k_page = common.k_slot = common.k_head = common.v_page = common.v_slot = common.v_head = 16;
  return attend_error(&common, T, Hq, R, max_new);
}

}  // namespace

extern "C" km_status kmeans_kv_append_form(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt, int64_t T,
                                           const void* q, int64_t q_heads, int64_t q_token, int64_t q_head,
                                           const void* k, int64_t k_token, int64_t k_head, const void* v,
                                           int64_t v_token, int64_t v_head, const float* q_weight,
                                           const float* k_weight, float eps, const km_kv_turn* turn,
                                           const int32_t* slots, void* q_out, int64_t o_token, int64_t o_head,
                                           void* stream) {
  const bool eight = scales != nullptr;
  if (const char* e = eight ? codes_error(cache, scales, true, v != nullptr) : cache_error(cache, v != nullptr))
    return invalid(e);
  if (eight && (!apart(cache, cache->k_page, cache->k_slot, cache->k_head) ||
                (v && !apart(cache, cache->v_page, cache->v_slot, cache->v_head))))
    return invalid("pages, slots and heads of an 8-bit cache must not overlap");
  if (eight && v && cache->k == cache->v) return invalid("keys and values of an 8-bit cache must be different arrays");
  if (const km_status s = dtype_error(dt)) return s;
  if (q_heads < 0 || q_heads > (1 << 20)) return invalid("q_heads must be 0 to 2^20");
  if (T < 0 || T > kMaxI) return invalid("T must be 0 to 2^31 - 1");
  if (T * (q_heads + 2 * cache->heads) > kMaxRows)
    return fail(KM_ERR_UNSUPPORTED, "T * (q_heads + 2 * heads) must be at most 2^28 - 16");
  // (a workgroup of the widest rows writes 16 tokens of a head: half a launch)
  if (eight && T * 2 * cache->heads > kMaxRows / 2)
    return fail(KM_ERR_UNSUPPORTED, "T * heads must be at most 2^26 - 4 with an 8-bit cache");
  if (!(eps >= 0.f)) return invalid("eps must not be negative");
  if (turn) {
    if (turn->rot < 16 || turn->rot > cache->dim || turn->rot % 16)
      return invalid("rot must be a multiple of 16 from 16 to the cache's dim");
    if (turn->max_pos < 1 || turn->max_pos > kMaxI) return invalid("max_pos must be 1 to 2^31 - 1");
    if (turn->axes < 1 || turn->axes > 4) return invalid("positions must have 1 to 4 axes");
    if (turn->axes > 1 && (turn->axis_stride < T || turn->axis_stride >= kMaxStride))
      return invalid("the rows of positions must not overlap (a stride of at least T, below 2^40)");
    if (!turn->rope || !aligned(turn->rope, 16)) return invalid("rope must be a 16-byte aligned pointer");
    if (!aligned(turn->positions, 4) || (T > 0 && !turn->positions))
      return invalid("positions must be a 4-byte aligned pointer");
    if (!aligned(turn->axis, 8)) return invalid("axis must be 8-byte aligned");
  }
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return invalid("q_weight and k_weight must be 16-byte aligned");
  if (!aligned(slots, 4)) return invalid("slots must be 4-byte aligned");
  if (T == 0) return KM_OK;
  if (q_heads > 0 && (!rows_ok(q, q_token, q_head) || !rows_ok(q_out, o_token, o_head)))
    return invalid("q and q_out must be 16-byte aligned with strides that are multiples of 8");
  if (!rows_ok(k, k_token, k_head)) return invalid("k must be 16-byte aligned with strides that are multiples of 8");
  if (v && !rows_ok(v, v_token, v_head))
    return invalid("v must be 16-byte aligned with strides that are multiples of 8");
  if (q_heads > 0 && q == q_out && (q_token != o_token || q_head != o_head))
    return invalid("q_out may be q itself only with the same strides");
  FormAppendArgs a = {};
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
  a.k8 = (uint8_t*)cache->k;
  a.v8 = (uint8_t*)cache->v;
  a.kc_page = cache->k_page;
  a.kc_slot = cache->k_slot;
  a.kc_head = cache->k_head;
  a.vc_page = cache->v_page;
  a.vc_slot = cache->v_slot;
  a.vc_head = cache->v_head;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.slots = slots;
  a.T = (int32_t)T;
  a.Hq = (int32_t)q_heads;
  a.Hkv = (int32_t)cache->heads;
  a.D = (int32_t)cache->dim;
  a.max_pos = 1;
  if (turn) {
    a.rope = turn->rope;
    a.positions = turn->positions;
    a.rot = (int32_t)turn->rot;
    a.max_pos = (int32_t)turn->max_pos;
    a.axis = turn->axis;
    a.axes = (int32_t)turn->axes;
    a.axis_stride = turn->axis_stride;
  }
  a.num_slots = (int32_t)(cache->pages * cache->page_size);
  a.page_shift = shift_of(cache->page_size);
  a.eps = eps;
  if (eight) {
    a.ks = scales->k;
    a.vs = scales->v;
    a.ks_page = scales->k_page;
    a.ks_head = scales->k_head;
    a.vs_page = scales->v_page;
    a.vs_head = scales->v_head;
  }
  return launched(launch_append_form(a, (int)dt, eight, turn && turn->interleaved != 0, (hipStream_t)stream));
}

extern "C" km_status kmeans_kv_read(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt,
                                    const int32_t* slots, int64_t n, void* k, int64_t k_row, int64_t k_head, void* v,
                                    int64_t v_row, int64_t v_head, void* stream) {
  if (!scales) return invalid("the scales are NULL");
  if (const char* e = codes_error(cache, scales, k != nullptr, v != nullptr)) return invalid(e);
  if (const km_status s = dtype_error(dt)) return s;
  if (n < 0 || n > kMaxI) return invalid("n must be 0 to 2^31 - 1");
  if (n * cache->heads > kMaxRows) return fail(KM_ERR_UNSUPPORTED, "n * heads must be at most 2^28 - 16");
  if (!aligned(slots, 4)) return invalid("slots must be 4-byte aligned");
  if (n == 0 || (!k && !v)) return KM_OK;
  if ((k && !rows_ok(k, k_row, k_head)) || (v && !rows_ok(v, v_row, v_head)))
    return invalid("k and v must be 16-byte aligned with strides that are multiples of 8");
  ReadArgs a = {};
  a.k = (const uint8_t*)cache->k;
  a.v = (const uint8_t*)cache->v;
  a.ks = scales->k;
  a.vs = scales->v;
  a.k_page = cache->k_page;
  a.k_slot = cache->k_slot;
  a.k_head = cache->k_head;
  a.v_page = cache->v_page;
  a.v_slot = cache->v_slot;
  a.v_head = cache->v_head;
  a.ks_page = scales->k_page;
  a.ks_head = scales->k_head;
  a.vs_page = scales->v_page;
  a.vs_head = scales->v_head;
  a.slots = slots;
  a.ko = (uint16_t*)k;
  a.vo = (uint16_t*)v;
  a.ko_row = k_row;
  a.ko_head = k_head;
  a.vo_row = v_row;
  a.vo_head = v_head;
  a.n = (int32_t)n;
  a.heads = (int32_t)cache->heads;
  a.D = (int32_t)cache->dim;
  a.num_slots = (int32_t)(cache->pages * cache->page_size);
  a.page_shift = shift_of(cache->page_size);
  return launched(launch_read(a, (int)dt, (hipStream_t)stream));
}

extern "C" size_t kmeans_kv_attend_form_workspace(const km_kv_cache* cache, const km_kv_scales* scales, int64_t T,
                                                  int64_t q_heads, int64_t R, int64_t max_new) {
  if (form_error(cache, scales, T, q_heads, R, max_new)) return 0;
  return std::max<size_t>(256, make_plan(T, q_heads, cache->heads, cache->dim, R, max_new).bytes);
}

extern "C" km_status kmeans_kv_attend_form(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt,
                                           const void* q, int64_t T, int64_t q_heads, int64_t q_token, int64_t q_head,
                                           const int32_t* block_table, int64_t R, int64_t width, int64_t table_stride,
                                           const int32_t* query_start, const int32_t* seq_lens,
                                           const float* log_weight, int64_t lw_page, int64_t lw_head,
                                           const km_kv_scores* scores, int64_t max_new, void* out, int64_t o_token,
                                           int64_t o_head, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (const char* e = form_error(cache, scales, T, q_heads, R, max_new)) return invalid(e);
  if (const km_status s = dtype_error(dt)) return s;
  if (!scores) return invalid("the scores are NULL");
  if (scores->window < 0 || scores->window > kMaxI) return invalid("window must be 0 (none) to 2^31 - 1");
  // (without weights the scores are in units of log 2)
  const float log2e = log_weight ? 1.f : 1.4426950408889634f;
  const float cap = scores->cap * log2e, unit = scores->cap > 0.f ? scores->scale / scores->cap : scores->scale * log2e;
  if (!(scores->cap >= 0.f) || !std::isfinite(cap))
    return invalid("cap must be 0 (none) or positive and finite, times log2(e) too");
  // (over the cap it is the factor of a tanh's argument, which is taken times 2 log2(e))
  if (!std::isfinite(scores->scale) || !std::isfinite(scores->cap > 0.f ? unit * (2.f * 1.4426950408889634f) : unit))
    return invalid("scale must be finite, times log2(e) and over cap (times 2 log2(e)) too");
  if (scores->cap > 0.f && scores->scale != 0.f && !(std::fabs(unit) >= 1.17549435e-38f))
    return invalid("scale / cap must not be below 2^-126");
  if (width < 0 || width > kMaxRoom / cache->page_size || table_stride < width || table_stride >= kMaxStride)
    return invalid("width must be at least 0, width * page_size at most 2^30 and table_stride at least width");
  if (!aligned(scores->slopes, 4) || !aligned(scores->prefix, 4))
    return invalid("slopes and prefix must be 4-byte aligned");
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
  FormArgs a = {};
  take_cache(a, cache, scales ? 1 : 2);
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.q_token = q_token;
  a.q_head = q_head;
  a.o_token = o_token;
  a.o_head = o_head;
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
  a.G = (int32_t)(q_heads / cache->heads);
  // A window of more than every position (at most 2^30) is none.
  a.window = scores->window >= kMaxRoom ? 0 : (int32_t)scores->window;
  a.scale = unit;
  a.cap = cap;
  a.slopes = scores->slopes;
  a.prefix = scores->prefix;
  if (scales) {
    a.ks = scales->k;
    a.vs = scales->v;
    a.ks_page = scales->k_page;
    a.ks_head = scales->k_head;
    a.vs_page = scales->v_page;
    a.vs_head = scales->v_head;
  }
  // most keys that a tile can see (a prefix may be as long as the room)
  const int64_t room = width * cache->page_size;
  const int64_t keys = std::max<int64_t>(
      1, a.window && !a.prefix ? std::min<int64_t>(room, a.window + max_new + 256) : room);
  const bool eight = scales != nullptr;
  const hipStream_t at = (hipStream_t)stream;
  return launched(attend_launches(
      a, p, keys, ws, log_weight != nullptr,
      [&](const FormArgs& x) { return (eight ? launch_decode_eight : launch_decode_form)(x, (int)dt, p.bm, at); },
      [&](const FormArgs& x) { return (eight ? launch_chunk_eight : launch_chunk_form)(x, (int)dt, at); },
      [&](const JoinArgs& x) { return launch_join_form(x, (int)dt, at); }));
}

extern "C" const char* kmeans_kv_form_last_error(void) { return g_error.c_str(); }

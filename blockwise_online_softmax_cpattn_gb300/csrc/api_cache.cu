// The C ABI of the 4-bit key/value cache: argument validation and dispatch.
#include <limits.h>
#include <math.h>

#include "api_internal.h"
#include "cache.cuh"

namespace cpattn {

static cpattn_status validate_cache(const cpattn_cache_desc* d, Cache* c) {
  if (!d) return CPATTN_ERR_INVALID_ARG;
  if (d->H_q <= 0 || d->H_kv <= 0 || d->D <= 0 || d->n_pages <= 0) return CPATTN_ERR_INVALID_ARG;
  if (d->H_q % d->H_kv) return CPATTN_ERR_INVALID_ARG;
  if (d->D != 64 && d->D != 128) return CPATTN_ERR_UNSUPPORTED;
  if ((d->group != 32 && d->group != 64 && d->group != 128) || d->group > d->D)
    return CPATTN_ERR_INVALID_ARG;
  if (d->page < kCacheTile || d->page % kCacheTile) return CPATTN_ERR_INVALID_ARG;
  if (d->dtype != CPATTN_F32 && d->dtype != CPATTN_BF16) return CPATTN_ERR_INVALID_ARG;
  if (d->o_dtype != CPATTN_F32 && d->o_dtype != d->dtype) return CPATTN_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) || !isfinite(d->scale)) return CPATTN_ERR_INVALID_ARG;
  if (d->causal != 0 && d->causal != 1) return CPATTN_ERR_INVALID_ARG;
  if (d->debug_fault < 0 || d->debug_fault > 3) return CPATTN_ERR_INVALID_ARG;
  if ((int64_t)d->n_pages * d->page > INT_MAX || d->H_q > 32767) return CPATTN_ERR_UNSUPPORTED;
  if (c) {
    c->Hq = d->H_q;
    c->Hkv = d->H_kv;
    c->D = d->D;
    c->G = d->group;
    c->page = d->page;
    c->n_pages = d->n_pages;
    c->bf16 = d->dtype == CPATTN_BF16;
    c->o_f32 = d->o_dtype == CPATTN_F32;
    c->causal = d->causal;
    c->scale = d->scale;
    c->debug_fault = d->debug_fault;
  }
  return CPATTN_OK;
}

// A request's tokens, the table's entries and what is counted over requests are kept in 32
// bits, with room for a page, a tile or a step of a loop behind the last one.
static bool lengths_fit(const Cache& c, int n_req, int max_pages) {
  return n_req <= (1 << 24) && (int64_t)n_req * max_pages <= INT_MAX && (int64_t)max_pages * c.page <= (1 << 30);
}

static bool aligned4(const void* p) { return p && ((uintptr_t)p % 4 == 0); }

// Strides keep every row on a 16-byte boundary; a stride may be 0 or negative for a
// dimension of extent 1 only, which any value suits.
static bool strides_ok(const Cache& c, int64_t tokens, int64_t heads, int64_t ts, int64_t hs) {
  const int64_t vec = c.bf16 ? 8 : 4;
  if (tokens > 1 && (ts < c.D || ts % vec)) return false;
  if (heads > 1 && (hs < c.D || hs % vec)) return false;
  return true;
}

}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cpattn_cache_bytes(const cpattn_cache_desc* desc) {
  Cache c;
  if (validate_cache(desc, &c) != CPATTN_OK) return 0;
  return (size_t)c.n_pages * c.Hkv * c.block_bytes();
}

size_t cpattn_cache_plan_workspace(const cpattn_cache_desc* desc, int n_req) {
  if (validate_cache(desc, nullptr) != CPATTN_OK || n_req < 0) return 0;
  return cache_plan_workspace(n_req);
}

cpattn_status cpattn_cache_plan(const cpattn_cache_desc* desc, int n_req, int max_pages,
                                const int32_t* len_old, const int32_t* len_new, int32_t* table,
                                int32_t* free_list, const int32_t* n_free, int32_t* n_free_out,
                                int32_t* len_out, int32_t* q_start, int32_t* slots, int n_slots,
                                void* workspace, size_t ws_bytes, void* stream) {
  Cache c;
  cpattn_status s = validate_cache(desc, &c);
  if (s != CPATTN_OK) return s;
  if (n_req < 1 || max_pages < 1 || n_slots < 0) return CPATTN_ERR_INVALID_ARG;
  if (!aligned4(len_old) || !aligned4(len_new) || !aligned4(table) || !aligned4(free_list) ||
      !aligned4(n_free) || !aligned4(n_free_out) || !aligned4(len_out) || !aligned4(q_start) ||
      (n_slots > 0 && !aligned4(slots)) || !aligned16(workspace))
    return CPATTN_ERR_INVALID_ARG;
  if (ws_bytes < cache_plan_workspace(n_req)) return CPATTN_ERR_INVALID_ARG;
  if (!lengths_fit(c, n_req, max_pages)) return CPATTN_ERR_UNSUPPORTED;
  PlanArgs a;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.page = c.page;
  a.n_pages = c.n_pages;
  a.n_slots = n_slots;
  a.len_old = len_old;
  a.len_new = len_new;
  a.table = table;
  a.free_list = free_list;
  a.n_free = n_free;
  a.n_free_out = n_free_out;
  a.len_out = len_out;
  a.q_start = q_start;
  a.slots = slots;
  a.ws = static_cast<int*>(workspace);
  cudaGetLastError();
  return from_cuda(launch_cache_plan(a, (cudaStream_t)stream));
}

cpattn_status cpattn_cache_append(const cpattn_cache_desc* desc, int n_tokens, const void* k,
                                  int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                  int64_t v_token_stride, int64_t v_head_stride,
                                  const int32_t* slots, void* cache, void* stream) {
  Cache c;
  cpattn_status s = validate_cache(desc, &c);
  if (s != CPATTN_OK) return s;
  if (n_tokens < 0) return CPATTN_ERR_INVALID_ARG;
  if (n_tokens == 0) return CPATTN_OK;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots) || !aligned16(cache) ||
      !strides_ok(c, n_tokens, c.Hkv, k_token_stride, k_head_stride) ||
      !strides_ok(c, n_tokens, c.Hkv, v_token_stride, v_head_stride))
    return CPATTN_ERR_INVALID_ARG;
  cudaGetLastError();
  return from_cuda(launch_cache_append(c, n_tokens, k, {k_token_stride, k_head_stride}, v,
                                       {v_token_stride, v_head_stride}, slots, cache, range_ptr(),
                                       (cudaStream_t)stream));
}

cpattn_status cpattn_cache_read(const cpattn_cache_desc* desc, int n_tokens, const int32_t* slots,
                                const void* cache, void* k, int64_t k_token_stride,
                                int64_t k_head_stride, void* v, int64_t v_token_stride,
                                int64_t v_head_stride, void* stream) {
  Cache c;
  cpattn_status s = validate_cache(desc, &c);
  if (s != CPATTN_OK) return s;
  if (n_tokens < 0) return CPATTN_ERR_INVALID_ARG;
  if (n_tokens == 0) return CPATTN_OK;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots) || !aligned16(cache) ||
      !strides_ok(c, n_tokens, c.Hkv, k_token_stride, k_head_stride) ||
      !strides_ok(c, n_tokens, c.Hkv, v_token_stride, v_head_stride))
    return CPATTN_ERR_INVALID_ARG;
  cudaGetLastError();
  return from_cuda(launch_cache_read(c, n_tokens, slots, cache, k, {k_token_stride, k_head_stride},
                                     v, {v_token_stride, v_head_stride}, (cudaStream_t)stream));
}

size_t cpattn_cache_attn_workspace(const cpattn_cache_desc* desc) {
  Cache c;
  if (validate_cache(desc, &c) != CPATTN_OK) return 0;
  return cache_attn_workspace(c);
}

cpattn_status cpattn_cache_attn(const cpattn_cache_desc* desc, int n_req, int max_pages,
                                int n_tokens, int max_q, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, const int32_t* q_start,
                                const int32_t* kv_len, const int32_t* table, const void* cache,
                                void* o, float* lse, void* workspace, size_t ws_bytes,
                                void* stream) {
  Cache c;
  cpattn_status s = validate_cache(desc, &c);
  if (s != CPATTN_OK) return s;
  if (n_req < 1 || max_pages < 1 || n_tokens < 0 || max_q < 1) return CPATTN_ERR_INVALID_ARG;
  if (n_tokens == 0) return CPATTN_OK;
  if (!aligned16(q) || !aligned4(q_start) || !aligned4(kv_len) || !aligned4(table) ||
      !aligned16(cache) || !aligned16(o) || (lse && !aligned4(lse)) || !aligned16(workspace) ||
      !strides_ok(c, n_tokens, c.Hq, q_token_stride, q_head_stride))
    return CPATTN_ERR_INVALID_ARG;
  if (ws_bytes < cache_attn_workspace(c)) return CPATTN_ERR_INVALID_ARG;
  if (!lengths_fit(c, n_req, max_pages) || (int64_t)n_tokens * c.Hq > INT_MAX)
    return CPATTN_ERR_UNSUPPORTED;
  CacheAttnArgs a;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.n_tokens = n_tokens;
  a.max_q = max_q;
  a.q = q;
  a.qs = {q_token_stride, q_head_stride};
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = table;
  a.cache = static_cast<const uint8_t*>(cache);
  a.o = o;
  a.lse = lse;
  a.ws = workspace;
  a.status = status_ptr();
  cudaGetLastError();
  return from_cuda(launch_cache_attn(c, a, (cudaStream_t)stream));
}

}  // extern "C"

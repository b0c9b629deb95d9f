// step_api.cpp -- host side of the verification step's operators declared in include/sfx.h: the
// 8-bit KV cache's write and read, the attention over it, and the verification of a draft.
//
// They need no context.  Host code checks the arguments it can see, derives the launch plan from
// the shapes alone (never from device memory) and enqueues kernels.
#include "../../include/sfx.h"
#include "errors.h"
#include "kv_attention.h"
#include "kv_cache.h"
#include "verify.h"

using namespace sfx;

namespace {

constexpr int64_t kMaxTokens = 0x7fffff00;  // positions and tile ends are int32
constexpr int64_t kMaxRows = 0x7fffffff;    // query rows of one call
constexpr int64_t kMaxThreads = 0xffffffff;  // of one launch: the runtime counts them in 32 bits
constexpr float kMaxScale = 0x1p64f;  // the softmax scale times a power of two in [2^-33, 2^30]
                                      // has to stay a normal number

using Wide = __int128;  // products of three 32-bit sizes

bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

int check_type(int32_t type, bool fp32) {
  if (type == SFX_TYPE_BF16 || type == SFX_TYPE_FP16 || (fp32 && type == SFX_TYPE_FP32))
    return SFX_OK;
  return fail(SFX_EINVAL, "element type %d is not supported here", type);
}

KvType kv_type(int32_t type) {
  return type == SFX_TYPE_FP16 ? kFp16 : (type == SFX_TYPE_FP32 ? kFp32 : kBf16);
}

// Checks the cache and the page table's width; fills the device view.
int check_cache(const sfx_kv_cache* c, int32_t B, int32_t T, int32_t max_pages,
                const int32_t* page_table, KvCache* out) {
  if (!c) return fail(SFX_EINVAL, "cache is NULL");
  if (B < 0 || T < 0 || max_pages < 0)
    return fail(SFX_EINVAL, "negative shape B=%d T=%d max_pages=%d", B, T, max_pages);
  if (c->num_pages < 0 || c->kv_heads < 1)
    return fail(SFX_EINVAL, "cache with num_pages=%d kv_heads=%d", c->num_pages, c->kv_heads);
  if (!dim_ok(c->head_dim))
    return fail(SFX_EINVAL, "head_dim=%d is not 64, 128 or 256", c->head_dim);
  if (c->page_size < kKvBlock || c->page_size > kKvMaxPage || c->page_size % kKvBlock)
    return fail(SFX_EINVAL, "page_size=%d is not a multiple of %d in [%d, %d]", c->page_size,
                kKvBlock, kKvBlock, kKvMaxPage);
  if ((int64_t)max_pages * c->page_size > kMaxTokens)
    return fail(SFX_ECAPACITY, "max_pages=%d of %d tokens pass 2^31 - 256 tokens", max_pages,
                c->page_size);
  if (B > 0 && T > 0 && max_pages > 0 && !page_table)
    return fail(SFX_EINVAL, "page_table is NULL");
  if (c->num_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale))
    return fail(SFX_EINVAL, "cache buffer is NULL");
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15)
    return fail(SFX_EINVAL, "cache codes must be aligned to 16 bytes");
  const int per_page = c->page_size / kKvBlock;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->heads = c->kv_heads;
  out->page_magic =
      per_page == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + per_page - 1) / per_page);
  out->k = (uint8_t*)c->k;
  out->v = (uint8_t*)c->v;
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  return SFX_OK;
}

KvStrides strides(const int64_t* s, int64_t T, int64_t heads, int64_t dim) {
  if (s) return KvStrides{s[0], s[1], s[2]};
  return KvStrides{T * heads * dim, heads * dim, dim};
}

int move_args(const sfx_kv_cache* cache, int32_t B, int32_t T, int32_t max_pages,
              const int32_t* page_table, const int32_t* start, const int32_t* count, void* k,
              const int64_t* k_strides, void* v, const int64_t* v_strides, int32_t type,
              KvMoveArgs* a) {
  int rc = check_cache(cache, B, T, max_pages, page_table, &a->c);
  if (!rc) rc = check_type(type, true);
  if (rc) return rc;
  if (B == 0 || T == 0) return SFX_OK;
  if (!start || !k || !v) return fail(SFX_EINVAL, "NULL array argument");
  if (kv_move_threads(B, T, cache->kv_heads) > kMaxThreads)
    return fail(SFX_ECAPACITY, "B=%d T=%d is too large for one call", B, T);
  a->B = B;
  a->T = T;
  a->max_pages = max_pages;
  a->page_table = page_table;
  a->start = start;
  a->count = count;
  a->k = k;
  a->v = v;
  a->ks = strides(k_strides, T, cache->kv_heads, cache->head_dim);
  a->vs = strides(v_strides, T, cache->kv_heads, cache->head_dim);
  return SFX_OK;
}

int attention_plan(const sfx_kv_cache* cache, int32_t B, int32_t T, int32_t q_heads,
                   int32_t max_pages, const int32_t* page_table, int32_t window, int32_t sinks,
                   KvAttentionArgs* a, size_t* bytes) {
  int rc = check_cache(cache, B, T, max_pages, page_table, &a->c);
  if (rc) return rc;
  if (q_heads < cache->kv_heads || q_heads % cache->kv_heads)
    return fail(SFX_EINVAL, "q_heads=%d is not a multiple of kv_heads=%d", q_heads,
                cache->kv_heads);
  if (window < 0 || sinks < 0)
    return fail(SFX_EINVAL, "negative window=%d or sinks=%d", window, sinks);
  a->B = B;
  a->T = T;
  a->group = q_heads / cache->kv_heads;
  a->max_pages = max_pages;
  a->page_table = page_table;
  a->window = window;
  a->sinks = sinks;
  if ((int64_t)T * a->group > (1 << 30) || Wide(B) * T * q_heads > kMaxRows)
    return fail(SFX_ECAPACITY, "B=%d T=%d q_heads=%d is too large for one call", B, T, q_heads);
  *bytes = kv_attention_plan(a, cache->head_dim);
  if (kv_attention_threads(*a) > kMaxThreads)
    return fail(SFX_ECAPACITY, "B=%d T=%d q_heads=%d is too large for one call", B, T, q_heads);
  return SFX_OK;
}

int verify_shape(int32_t B, int32_t k, int32_t V, int32_t type, VerifyArgs* a, size_t* bytes) {
  int rc = check_type(type, true);
  if (rc) return rc;
  if (B < 0) return fail(SFX_EINVAL, "negative B=%d", B);
  if (k < 0 || k > 32) return fail(SFX_EINVAL, "k=%d outside [0,32]", k);
  if (V < 1 || V > (1 << 30)) return fail(SFX_EINVAL, "V=%d outside [1,2^30]", V);
  a->B = B;
  a->k = k;
  a->V = V;
  *bytes = verify_plan(a, kv_type(type));
  if (verify_threads(*a) > kMaxThreads)
    return fail(SFX_ECAPACITY, "B=%d k=%d V=%d is too large for one call", B, k, V);
  return SFX_OK;
}

}  // namespace

extern "C" {

int sfx_kv_write(const sfx_kv_cache* cache, int32_t B, int32_t T, int32_t max_pages,
                 const int32_t* page_table, const int32_t* start, const int32_t* count,
                 const void* k, const int64_t* k_strides, const void* v,
                 const int64_t* v_strides, int32_t type, void* stream) {
  KvMoveArgs a{};
  int rc = move_args(cache, B, T, max_pages, page_table, start, count, const_cast<void*>(k),
                     k_strides, const_cast<void*>(v), v_strides, type, &a);
  if (rc || a.B == 0 || cache->num_pages == 0 || max_pages == 0) return rc;
  HIP_OR_RETURN(launch_kv_write(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                "kv write launch");
  return SFX_OK;
}

int sfx_kv_read(const sfx_kv_cache* cache, int32_t B, int32_t T, int32_t max_pages,
                const int32_t* page_table, const int32_t* start, const int32_t* count, void* k,
                const int64_t* k_strides, void* v, const int64_t* v_strides, int32_t type,
                void* stream) {
  KvMoveArgs a{};
  int rc = move_args(cache, B, T, max_pages, page_table, start, count, k, k_strides, v,
                     v_strides, type, &a);
  if (rc || a.B == 0) return rc;
  HIP_OR_RETURN(launch_kv_read(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                "kv read launch");
  return SFX_OK;
}

int sfx_kv_attention_workspace_bytes(const sfx_kv_cache* cache, int32_t B, int32_t T,
                                     int32_t q_heads, int32_t max_pages, int32_t window,
                                     int32_t sinks, size_t* bytes) {
  if (!bytes) return fail(SFX_EINVAL, "bytes is NULL");
  KvAttentionArgs a{};
  static const int32_t none = 0;  // the plan does not look at the table
  return attention_plan(cache, B, T, q_heads, max_pages, &none, window, sinks, &a, bytes);
}

int sfx_kv_attention(const sfx_kv_cache* cache, int32_t B, int32_t T, int32_t q_heads,
                     int32_t max_pages, const int32_t* page_table, const int32_t* seq_lens,
                     const int32_t* q_lens, const void* q, const int64_t* q_strides, void* out,
                     int32_t type, float scale, int32_t window, int32_t sinks, void* workspace,
                     size_t workspace_bytes, void* stream) {
  KvAttentionArgs a{};
  size_t bytes = 0;
  int rc = attention_plan(cache, B, T, q_heads, max_pages, page_table, window, sinks, &a, &bytes);
  if (!rc) rc = check_type(type, false);
  if (rc) return rc;
  if (!(scale >= 1.f / kMaxScale && scale <= kMaxScale))
    return fail(SFX_EINVAL, "scale=%g outside [2^-64, 2^64]", (double)scale);
  if (B == 0 || T == 0) return SFX_OK;
  if (!seq_lens || !q || !out) return fail(SFX_EINVAL, "NULL array argument");
  if ((uintptr_t)out & 15) return fail(SFX_EINVAL, "out must be aligned to 16 bytes");
  if (bytes > 0 && (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)))
    return fail(SFX_EINVAL, "workspace of %zu bytes (16-byte aligned) needed, %zu given", bytes,
                workspace ? workspace_bytes : (size_t)0);
  a.seq_lens = seq_lens;
  a.q_lens = q_lens;
  a.q = q;
  a.qs = strides(q_strides, T, q_heads, cache->head_dim);
  a.out = out;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (bytes > 0) kv_attention_place(&a, cache->head_dim, workspace);
  HIP_OR_RETURN(launch_kv_attention(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                "kv attention launch");
  return SFX_OK;
}

int sfx_verify_workspace_bytes(int32_t B, int32_t k, int32_t V, int32_t type, size_t* bytes) {
  if (!bytes) return fail(SFX_EINVAL, "bytes is NULL");
  VerifyArgs a{};
  return verify_shape(B, k, V, type, &a, bytes);
}

int sfx_verify(int32_t B, int32_t k, int32_t V, const void* logits, int64_t batch_stride,
               int64_t slot_stride, int32_t type, const float* temperature, const int32_t* draft,
               const int32_t* num_valid, const float* u_accept, const float* u_sample,
               int32_t* sampled, int32_t* num_accepted, void* workspace, size_t workspace_bytes,
               void* stream) {
  VerifyArgs a{};
  size_t bytes = 0;
  int rc = verify_shape(B, k, V, type, &a, &bytes);
  if (rc || B == 0) return rc;
  if (!logits || !u_sample || !sampled || !num_accepted || (k > 0 && (!draft || !u_accept)))
    return fail(SFX_EINVAL, "NULL array argument");
  if (bytes > 0 && (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)))
    return fail(SFX_EINVAL, "workspace of %zu bytes (16-byte aligned) needed, %zu given", bytes,
                workspace ? workspace_bytes : (size_t)0);
  a.logits = logits;
  a.batch_stride = batch_stride;
  a.slot_stride = slot_stride;
  a.temperature = temperature;
  a.draft = draft;
  a.num_valid = num_valid;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.sampled = sampled;
  a.num_accepted = num_accepted;
  verify_place(&a, workspace);
  HIP_OR_RETURN(launch_verify(a, kv_type(type), (hipStream_t)stream), "verify launch");
  return SFX_OK;
}

}  // extern "C"

// step_api.cpp -- host side of the verification step's operators declared in include/sfx.h: the
// 8-bit KV cache's writes and read, the attention over it, the verification of a draft, and what a
// packed batch needs besides: pages, the batch's layout and the attention of prompts.
//
// They need no context.  Host code checks the arguments it can see, derives the launch plan from
// the shapes alone (never from device memory) and enqueues kernels.
#include "../../include/sfx.h"

#include <initializer_list>

#include "errors.h"
#include "kv_attention.h"
#include "kv_cache.h"
#include "pages.h"
#include "tile_attention.h"
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

KvStrides packed_strides(const int64_t* s, int64_t heads, int64_t dim) {
  if (s) return KvStrides{0, s[0], s[1]};
  return KvStrides{0, heads * dim, dim};
}

int check_heads(int32_t q_heads, int32_t kv_heads, int32_t window, int32_t sinks) {
  if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads)
    return fail(SFX_EINVAL, "q_heads=%d is not a multiple of kv_heads=%d", q_heads, kv_heads);
  if (window < 0 || sinks < 0)
    return fail(SFX_EINVAL, "negative window=%d or sinks=%d", window, sinks);
  return SFX_OK;
}

// The plan of an attention of packed rows; a->c is filled for one over the cache.
int tile_plan(int32_t B, int32_t N, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
              int32_t window, int32_t sinks, bool paged, TileAttentionArgs* a, size_t* bytes) {
  a->B = B;
  a->N = N;
  a->heads = kv_heads;
  a->group = q_heads / kv_heads;
  a->window = window;
  a->sinks = sinks;
  if (Wide(N) * q_heads > kMaxRows || B > (1 << 24))
    return fail(SFX_ECAPACITY, "B=%d N=%d q_heads=%d is too large for one call", B, N, q_heads);
  *bytes = tile_attention_plan(a, head_dim, paged);
  if (tile_attention_threads(*a, head_dim) > kMaxThreads)
    return fail(SFX_ECAPACITY, "B=%d N=%d q_heads=%d is too large for one call", B, N, q_heads);
  return SFX_OK;
}

// Requests of at most this many rows (tokens x query heads of a group) go to the kernel whose
// wavefronts share out the tokens instead of the rows.  16 requests of 8192 tokens, 8 cached heads of
// 128: with 192 rows each it takes 150 us and the other kernel, tiles of 256 rows, 184; with 256 rows
// 255 and 193.
constexpr int kFewRows = 192;

struct PackedArgs {
  KvAttentionArgs few;  // requests of few rows; few.T == 0: none
  TileAttentionArgs many;
  bool has_many;
};

int packed_plan(const sfx_kv_cache* cache, int32_t B, int32_t N, int32_t max_q, int32_t q_heads,
                int32_t max_pages, const int32_t* page_table, int32_t window, int32_t sinks,
                PackedArgs* p, size_t* bytes) {
  TileAttentionArgs& m = p->many;
  int rc = check_cache(cache, B, N, max_pages, page_table, &m.c);
  if (!rc) rc = check_heads(q_heads, cache->kv_heads, window, sinks);
  if (rc) return rc;
  if (max_q < 0) return fail(SFX_EINVAL, "negative max_q=%d", max_q);
  if (Wide(N) * q_heads > kMaxRows || B > (1 << 24))
    return fail(SFX_ECAPACITY, "B=%d N=%d q_heads=%d is too large for one call", B, N, q_heads);
  m.max_pages = cache->num_pages > 0 ? max_pages : 0;  // no pages: no tokens
  m.max_q = max_q < N ? max_q : N;
  m.page_table = page_table;
  const int group = q_heads / cache->kv_heads;
  int few = kFewRows / group;
  few = few < m.max_q ? few : m.max_q;
  if (B == 0 || N == 0) few = 0;
  m.few = few;
  p->has_many = m.max_q > few || few == 0;
  size_t few_bytes = 0, many_bytes = 0;
  if (p->has_many)
    rc = tile_plan(B, N, q_heads, cache->kv_heads, cache->head_dim, window, sinks, true, &m,
                   &many_bytes);
  if (!rc && few > 0) {
    rc = attention_plan(cache, B, few, q_heads, max_pages, page_table, window, sinks, &p->few,
                        &few_bytes);
    p->few.N = N;
    p->few.max_q = m.max_q;
    p->few.zero = !p->has_many;
  }
  // one after the other on one stream: they share the workspace
  *bytes = few_bytes > many_bytes ? few_bytes : many_bytes;
  return rc;
}

int prompt_plan(int32_t B, int32_t N, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                int32_t window, int32_t sinks, TileAttentionArgs* a, size_t* bytes) {
  if (B < 0 || N < 0) return fail(SFX_EINVAL, "negative shape B=%d N=%d", B, N);
  if (!dim_ok(head_dim)) return fail(SFX_EINVAL, "head_dim=%d is not 64, 128 or 256", head_dim);
  int rc = check_heads(q_heads, kv_heads, window, sinks);
  if (rc) return rc;
  return tile_plan(B, N, q_heads, kv_heads, head_dim, window, sinks, false, a, bytes);
}

// What both attentions of packed rows check beyond the plan.
int check_rows(int32_t N, const int32_t* offsets, const void* q, const void* out, int32_t type,
               float scale, size_t bytes, const void* workspace, size_t workspace_bytes) {
  int rc = check_type(type, false);
  if (rc) return rc;
  if (!(scale >= 1.f / kMaxScale && scale <= kMaxScale))
    return fail(SFX_EINVAL, "scale=%g outside [2^-64, 2^64]", (double)scale);
  if (N == 0) return SFX_OK;
  if (!offsets || !q || !out) return fail(SFX_EINVAL, "NULL array argument");
  if ((uintptr_t)out & 15) return fail(SFX_EINVAL, "out must be aligned to 16 bytes");
  if (bytes > 0 && (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)))
    return fail(SFX_EINVAL, "workspace of %zu bytes (16-byte aligned) needed, %zu given", bytes,
                workspace ? workspace_bytes : (size_t)0);
  return SFX_OK;
}

// Whether rows x heads of `dim` 16-bit values share memory with [lo, hi).
bool rows_meet(const void* p, KvStrides s, int64_t rows, int64_t heads, int64_t dim, Wide lo,
               Wide hi) {
  Wide row = Wide(s.token) * 2, head = Wide(s.head) * 2, base = (uintptr_t)p, size = dim * 2;
  if (s.head == dim) {  // a row's heads are one piece
    size *= heads;
    heads = 1;
  }
  if (row < 0) {
    base += (rows - 1) * row;
    row = -row;
  }
  if (head < 0) {
    base += (heads - 1) * head;
    head = -head;
  }
  if (lo >= base + (rows - 1) * row + (heads - 1) * head + size || hi <= base) return false;
  for (int64_t h = 0; h < heads; ++h, base += head) {
    // the first row that ends behind lo
    const Wide past = lo - size - base, t = past < 0 || row == 0 ? 0 : past / row + 1;
    if (t < rows && base + t * row < hi && base + t * row + size > lo) return true;
  }
  return false;
}

// out, dense, over the rows of an input: they are stored while other workgroups still read.  Only a
// query's own place may take its result: its reader is the workgroup that stores it, or is done.
int check_out(const void* out, int64_t N, int64_t q_heads, int64_t dim, const char* name,
              const void* p, KvStrides s, int64_t heads, bool query) {
  if (query && p == out && (s.head == dim || heads == 1) && (s.token == heads * dim || N == 1))
    return SFX_OK;
  const Wide lo = (uintptr_t)out;
  if (rows_meet(p, s, N, heads, dim, lo, lo + Wide(N) * q_heads * dim * 2))
    return fail(SFX_EINVAL, "out and %s share memory", name);
  return SFX_OK;
}

// The fields that both kernels' arguments have.
template <typename Args>
void fill_rows(Args* a, const int32_t* offsets, const void* q, KvStrides qs, void* out,
               float scale) {
  a->offsets = offsets;
  a->q = q;
  a->qs = qs;
  a->out = out;
  a->scale_log2 = scale * 1.4426950408889634f;
}

// An array of a call, as long as the call may read or write it.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};

// The first `written` of the arrays are written: they share no memory with any other.  Workgroups
// read the inputs at any time, also after others have stored their outputs.
int check_apart(std::initializer_list<Span> arrays, int written) {
  const Span* s = arrays.begin();
  const int n = (int)arrays.size();
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j) {
      const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[j].p;
      if (a && b && s[i].bytes && s[j].bytes && a < b + s[j].bytes && b < a + s[i].bytes)
        return fail(SFX_EINVAL, "%s and %s share memory", s[i].name, s[j].name);
    }
  return SFX_OK;
}

int check_pages(int32_t B, int32_t max_pages, int32_t page_size, int32_t num_pages) {
  if (B < 0 || max_pages < 0 || num_pages < 0)
    return fail(SFX_EINVAL, "negative shape B=%d max_pages=%d num_pages=%d", B, max_pages,
                num_pages);
  if (page_size < 1) return fail(SFX_EINVAL, "page_size=%d is not positive", page_size);
  // workgroups count requests in steps of 1024, in 32 bits
  if (B > 0x7fffffff - 1023) return fail(SFX_ECAPACITY, "B=%d is too large for one call", B);
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

int sfx_pages_reserve_workspace_bytes(int32_t B, int32_t max_pages, size_t* bytes) {
  if (!bytes) return fail(SFX_EINVAL, "bytes is NULL");
  int rc = check_pages(B, max_pages, 1, 0);
  if (rc) return rc;
  if ((int64_t)B * max_pages > kMaxRows)
    return fail(SFX_ECAPACITY, "B=%d max_pages=%d is too large for one call", B, max_pages);
  *bytes = reserve_plan_words(B, max_pages) * sizeof(int32_t);
  return SFX_OK;
}

int sfx_pages_reserve(int32_t B, int32_t max_pages, int32_t page_size, int32_t num_pages,
                      const int32_t* tokens, int32_t* page_table, int32_t* held,
                      int32_t* free_pages, int32_t* num_free, int32_t* missing, void* workspace,
                      size_t workspace_bytes, void* stream) {
  size_t bytes = 0;
  int rc = check_pages(B, max_pages, page_size, num_pages);
  if (!rc) rc = sfx_pages_reserve_workspace_bytes(B, max_pages, &bytes);
  if (rc || B == 0) return rc;
  if (!tokens || !held || !num_free || (max_pages > 0 && !page_table) ||
      (num_pages > 0 && !free_pages))
    return fail(SFX_EINVAL, "NULL array argument");
  if (bytes > 0 && (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)))
    return fail(SFX_EINVAL, "workspace of %zu bytes (16-byte aligned) needed, %zu given", bytes,
                workspace ? workspace_bytes : (size_t)0);
  const size_t b = (size_t)B * 4;
  // missing in the place of tokens is fine: the thread that writes one is the last to read the other
  const int32_t* miss = missing == tokens ? nullptr : missing;
  rc = check_apart({{"page_table", page_table, b * max_pages}, {"held", held, b},
                    {"free_pages", free_pages, (size_t)num_pages * 4}, {"num_free", num_free, 4},
                    {"missing", miss, b}, {"workspace", workspace, bytes}, {"tokens", tokens, b}},
                   6);
  if (rc) return rc;
  const ReserveArgs a{B,    max_pages,  page_size, num_pages, tokens, page_table,
                      held, free_pages, num_free,  missing,   (int32_t*)workspace};
  HIP_OR_RETURN(launch_reserve(a, (hipStream_t)stream), "pages reserve launch");
  return SFX_OK;
}

int sfx_step_layout(int32_t B, int32_t N, int32_t max_pages, int32_t page_size, int32_t num_pages,
                    const int32_t* page_table, const int32_t* start, const int32_t* count,
                    int32_t* offsets, int32_t* seq_lens, int32_t* request, int32_t* position,
                    int64_t* slots, void* stream) {
  int rc = check_pages(B, max_pages, page_size, num_pages);
  if (rc) return rc;
  if (N < 0) return fail(SFX_EINVAL, "negative N=%d", N);
  if (!offsets || (B > 0 && (!start || !count || (slots && max_pages > 0 && !page_table))))
    return fail(SFX_EINVAL, "NULL array argument");
  if (layout_threads(N) > kMaxThreads)
    return fail(SFX_ECAPACITY, "N=%d is too large for one call", N);
  const size_t b = (size_t)B * 4, n = (size_t)N;
  rc = check_apart({{"offsets", offsets, b + 4}, {"seq_lens", seq_lens, b},
                    {"request", request, n * 4}, {"position", position, n * 4},
                    {"slots", slots, n * 8}, {"start", start, b}, {"count", count, b},
                    {"page_table", slots ? page_table : nullptr, b * max_pages}},
                   5);
  if (rc) return rc;
  const LayoutArgs a{B,     N,       max_pages, page_size, num_pages, page_table, start,
                     count, offsets, seq_lens,  request,   position,  slots};
  HIP_OR_RETURN(launch_layout(a, (hipStream_t)stream), "step layout launch");
  return SFX_OK;
}

int sfx_kv_write_slots(const sfx_kv_cache* cache, int32_t N, const int64_t* slots, const void* k,
                       const int64_t* k_strides, const void* v, const int64_t* v_strides,
                       int32_t type, void* stream) {
  KvSlotArgs a{};
  int rc = check_cache(cache, 0, N, 0, nullptr, &a.c);
  if (!rc) rc = check_type(type, true);
  if (rc || N == 0) return rc;
  if (!slots || !k || !v) return fail(SFX_EINVAL, "NULL array argument");
  a.N = N;
  a.window = kv_slot_window(N, cache->kv_heads);
  if (kv_slot_threads(N, a.window, cache->kv_heads) > kMaxThreads)
    return fail(SFX_ECAPACITY, "N=%d is too large for one call", N);
  a.slots = slots;
  a.k = k;
  a.v = v;
  a.ks = packed_strides(k_strides, cache->kv_heads, cache->head_dim);
  a.vs = packed_strides(v_strides, cache->kv_heads, cache->head_dim);
  if (cache->num_pages == 0) return SFX_OK;
  HIP_OR_RETURN(launch_kv_write_slots(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                "kv write launch");
  return SFX_OK;
}

int sfx_kv_attention_packed_workspace_bytes(const sfx_kv_cache* cache, int32_t B, int32_t N,
                                            int32_t max_q, int32_t q_heads, int32_t max_pages,
                                            int32_t window, int32_t sinks, size_t* bytes) {
  if (!bytes) return fail(SFX_EINVAL, "bytes is NULL");
  PackedArgs p{};
  static const int32_t none = 0;  // the plan does not look at the table
  return packed_plan(cache, B, N, max_q, q_heads, max_pages, &none, window, sinks, &p, bytes);
}

int sfx_kv_attention_packed(const sfx_kv_cache* cache, int32_t B, int32_t N, int32_t max_q,
                            int32_t q_heads, int32_t max_pages, const int32_t* page_table,
                            const int32_t* seq_lens, const int32_t* offsets, const void* q,
                            const int64_t* q_strides, void* out, int32_t type, float scale,
                            int32_t window, int32_t sinks, void* workspace,
                            size_t workspace_bytes, void* stream) {
  PackedArgs p{};
  size_t bytes = 0;
  int rc = packed_plan(cache, B, N, max_q, q_heads, max_pages, page_table, window, sinks, &p,
                       &bytes);
  if (!rc) rc = check_rows(N, offsets, q, out, type, scale, bytes, workspace, workspace_bytes);
  if (rc || N == 0) return rc;
  if (B > 0 && !seq_lens) return fail(SFX_EINVAL, "NULL array argument");
  const KvStrides qs = packed_strides(q_strides, q_heads, cache->head_dim);
  rc = check_out(out, N, q_heads, cache->head_dim, "q", q, qs, q_heads, true);
  if (rc) return rc;
  if (p.has_many) {
    TileAttentionArgs& a = p.many;
    fill_rows(&a, offsets, q, qs, out, scale);
    a.seq_lens = seq_lens;
    if (a.splits > 1) tile_attention_place(&a, cache->head_dim, workspace);
    HIP_OR_RETURN(launch_chunk_attention(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                  "packed attention launch");
  }
  if (p.few.T > 0) {
    KvAttentionArgs& a = p.few;
    fill_rows(&a, offsets, q, qs, out, scale);
    a.seq_lens = seq_lens;
    if (a.splits > 1) kv_attention_place(&a, cache->head_dim, workspace);
    HIP_OR_RETURN(launch_kv_attention(a, cache->head_dim, kv_type(type), (hipStream_t)stream),
                  "packed attention launch");
  }
  return SFX_OK;
}

int sfx_prompt_attention_workspace_bytes(int32_t B, int32_t N, int32_t q_heads, int32_t kv_heads,
                                         int32_t head_dim, int32_t window, int32_t sinks,
                                         size_t* bytes) {
  if (!bytes) return fail(SFX_EINVAL, "bytes is NULL");
  TileAttentionArgs a{};
  return prompt_plan(B, N, q_heads, kv_heads, head_dim, window, sinks, &a, bytes);
}

int sfx_prompt_attention(int32_t B, int32_t N, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                         const int32_t* offsets, const void* q, const int64_t* q_strides,
                         const void* k, const int64_t* k_strides, const void* v,
                         const int64_t* v_strides, void* out, int32_t type, float scale,
                         int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                         void* stream) {
  TileAttentionArgs a{};
  size_t bytes = 0;
  int rc = prompt_plan(B, N, q_heads, kv_heads, head_dim, window, sinks, &a, &bytes);
  if (!rc) rc = check_rows(N, offsets, q, out, type, scale, bytes, workspace, workspace_bytes);
  if (rc || N == 0) return rc;
  if (!k || !v) return fail(SFX_EINVAL, "NULL array argument");
  fill_rows(&a, offsets, q, packed_strides(q_strides, q_heads, head_dim), out, scale);
  if (bytes > 0) tile_attention_place(&a, head_dim, workspace);
  a.k = k;
  a.v = v;
  a.ks = packed_strides(k_strides, kv_heads, head_dim);
  a.vs = packed_strides(v_strides, kv_heads, head_dim);
  rc = check_out(out, N, q_heads, head_dim, "q", q, a.qs, q_heads, true);
  if (!rc) rc = check_out(out, N, q_heads, head_dim, "k", k, a.ks, kv_heads, false);
  if (!rc) rc = check_out(out, N, q_heads, head_dim, "v", v, a.vs, kv_heads, false);
  if (rc) return rc;
  HIP_OR_RETURN(launch_prompt_attention(a, head_dim, kv_type(type), (hipStream_t)stream),
                "prompt attention launch");
  return SFX_OK;
}

}  // extern "C"

// kv_attention.h -- launch interface of the attention over the 8-bit cache (internal to libsfx).
#pragma once

#include "kv_cache.h"

namespace sfx {

struct KvAttentionArgs {
  KvCache c;
  int32_t B, T, group, max_pages;  // group: query heads per cached head
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_lens;  // NULL: T for every request
  const void* q;
  KvStrides qs;
  void* out;              // [B, T, heads * group, dim]
  float scale_log2;       // softmax scale * log2(e)
  int32_t window, sinks;  // window 0: no window
  // plan (kv_attention_plan)
  int32_t chunks;           // workgroups over the rows of one request and head
  int32_t splits;           // workgroups over the tokens
  int32_t tiles_per_split;  // 32-token tiles of one split
  float* part_o;            // [splits][B * heads * T * group][dim]  (splits > 1)
  float2* part_ml;          // [splits][B * heads * T * group]: maximum, sum
};

// Fills the plan from the shapes; returns the workspace bytes it needs.
size_t kv_attention_plan(KvAttentionArgs* a, int dim);

// Threads of the planned launch (the join has fewer: calls that split have few rows).
int64_t kv_attention_threads(const KvAttentionArgs& a);

// Places the plan's buffers in the workspace.
void kv_attention_place(KvAttentionArgs* a, int dim, void* workspace);

hipError_t launch_kv_attention(const KvAttentionArgs& a, int dim, KvType type, hipStream_t st);

}  // namespace sfx

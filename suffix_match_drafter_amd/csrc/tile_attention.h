// tile_attention.h -- launch interface of the attention of many rows: whole prompts over their own
// keys and values, and packed chunks over the 8-bit cache (internal to libsfx).
#pragma once

#include "kv_cache.h"

namespace sfx {

struct TileAttentionArgs {
  int32_t B, N, heads, group;  // heads: of keys and values; group: query heads of each
  const int32_t* offsets;      // [B + 1]
  const void* q;               // [N, heads * group, dim]; strides[batch] is not used
  KvStrides qs;
  void* out;                   // the same shape, dense
  float scale_log2;            // softmax scale * log2(e)
  int32_t window, sinks;       // window 0: no window
  // prompts: keys and values [N, heads, dim]
  const void* k;
  const void* v;
  KvStrides ks, vs;
  // chunks: the cache
  KvCache c;
  int32_t max_pages, max_q;    // rows of a request from max_q on are zero
  int32_t few;                 // requests of 1 to `few` rows (tokens) are another call's
  const int32_t* page_table;
  const int32_t* seq_lens;
  // plan (tile_attention_plan)
  int32_t splits;              // workgroups over the tokens of one tile of rows
  int32_t least;               // token tiles that a split has at least
  float* part_o;               // [splits][N * heads * group][dim]  (splits > 1)
  float2* part_ml;             // [splits][N * heads * group]: maximum, sum
};

// Fills the plan from the shapes; returns the workspace bytes it needs.
size_t tile_attention_plan(TileAttentionArgs* a, int dim, bool paged);

// Threads of the planned launch, the larger of its two.
__int128 tile_attention_threads(const TileAttentionArgs& a, int dim);

// Places the plan's buffers in the workspace.
void tile_attention_place(TileAttentionArgs* a, int dim, void* workspace);

hipError_t launch_prompt_attention(const TileAttentionArgs& a, int dim, KvType type, hipStream_t st);
hipError_t launch_chunk_attention(const TileAttentionArgs& a, int dim, KvType type, hipStream_t st);

}  // namespace sfx

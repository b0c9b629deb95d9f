// kv_cache.h -- the paged 8-bit KV cache as its kernels see it (internal to libsfx).
//
// A page holds page_size tokens of every head.  Keys and values are e4m3 codes with one
// power-of-two scale per block of 32 tokens, head and tensor; a stored value is code * scale.
// Both tensors lie in the order in which the attention's matrix instructions take them, so a
// wavefront reads them with whole-kilobyte loads straight into its operand registers:
//
//   keys    [page][head][dim/64][token][64]: 16 tokens of one 64-dim slab are 1 KB;
//   values  [page][head][block][dim/32][r 16][g 4][f 2][j 2][i 4]: token 16 j + 4 g + i of the
//           block, dim 32 slab + 2 r + f.  16 bytes are two adjacent dims of the 8 tokens whose
//           probabilities one lane of the score product holds (see kv_attention.hip), so the
//           values need no transposition and the probabilities no exchange between lanes;
//   scales  [page][head][block] float32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfx {

constexpr int kKvBlock = 32;     // tokens per scale
constexpr int kKvMaxPage = 2048;
constexpr int kKvMinExp = -32;   // block scales lie in [2^-32, 2^31]: the ratio of any two blocks
constexpr int kKvMaxExp = 31;    // then keeps the attention's fp32 sums within range

struct KvCache {
  int32_t num_pages, page_size, heads;
  uint32_t page_magic;  // ceil(2^32 / blocks per page): block -> page by one multiplication
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
};

enum KvType { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

struct KvStrides {  // elements; the dims of one head are contiguous
  int64_t batch, token, head;
};

struct KvMoveArgs {
  KvCache c;
  int32_t B, T, max_pages;
  const int32_t* page_table;
  const int32_t* start;
  const int32_t* count;
  void* k;  // read by the write, written by the read
  void* v;
  KvStrides ks, vs;
};

constexpr int kKvMoveWaves = 4;  // wavefronts of a workgroup of the write and the read

// Blocks that T tokens can touch, whatever the start.
inline int64_t kv_blocks_of(int T) { return ((int64_t)T + kKvBlock - 2) / kKvBlock + 1; }

// Threads of a write's or read's launch: one wavefront per (request, block, tensor, head).
inline __int128 kv_move_threads(int B, int T, int heads) {
  const __int128 units = __int128(B) * kv_blocks_of(T) * 2 * heads;
  return (units + kKvMoveWaves - 1) / kKvMoveWaves * (64 * kKvMoveWaves);
}

// The write of a packed batch by slots; strides[batch] is not used.
struct KvSlotArgs {
  KvCache c;
  int32_t N, window;  // tokens, and how many of them one wavefront looks at (1..32)
  const int64_t* slots;
  const void* k;
  const void* v;
  KvStrides ks, vs;
};

// Tokens a wavefront looks at: as many as leave 8192 wavefronts, the card's fill.  In prompts only one
// of 32 tokens starts a block, so wavefronts of few tokens mostly find nothing (18432 tokens of prompts,
// 8 heads of 128 in bf16: a call of 113 us with one token each, 41 with 8, 24 to 27 with 32); where
// every token starts one, a wavefront of many works on one after the other (256 single tokens: 9 us
// with one token each, 25 with 8, 85 with 32).
inline int32_t kv_slot_window(int64_t N, int64_t heads) {
  const int64_t w = N * heads / 4096;
  return w < 1 ? 1 : (w > 32 ? 32 : (int32_t)w);
}

inline __int128 kv_slot_threads(int64_t N, int64_t window, int64_t heads) {
  const __int128 units = __int128((N + window - 1) / window) * 2 * heads;
  return (units + kKvMoveWaves - 1) / kKvMoveWaves * (64 * kKvMoveWaves);
}

hipError_t launch_kv_write_slots(const KvSlotArgs& a, int dim, KvType type, hipStream_t st);

hipError_t launch_kv_write(const KvMoveArgs& a, int dim, KvType type, hipStream_t st);
hipError_t launch_kv_read(const KvMoveArgs& a, int dim, KvType type, hipStream_t st);

// ---------------------------------------------------------------- device helpers
// Page of a 32-token block within its request: block / (page_size / 32).  With n <= 64 blocks a page
// the magic is too large by less than n / 2^32 of itself, which over blocks below 2^26 adds less
// than (n - 1) / n 2^-6 to the quotient: not enough to pass the next page, 1 / n >= 2^-6 away.
__device__ __forceinline__ int kv_page_of(const KvCache& c, int block) {
  return c.page_magic ? (int)__umulhi((unsigned)block, c.page_magic) : block;
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float kv_pow2(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of a stored scale, whatever the memory holds.
__device__ __forceinline__ int kv_exp_of(float scale) {
  const int e = ((__float_as_int(scale) >> 23) & 255) - 127;
  return e < kKvMinExp ? kKvMinExp : (e > kKvMaxExp ? kKvMaxExp : e);
}

}  // namespace sfx

// kv_attention.hip -- attention of a request's newest tokens over its paged 8-bit cache.
//
// Row t of the q_len newest tokens stands at position p = seq_len - q_len + t and sees the tokens
// j <= p with, under a window, p - window < j or j < sinks:
//   out_t = sum_j softmax_j(scale q_t . k_j) v_j,    zero for a row that sees nothing.
//
// Decomposition.  The rows of one request and cached head (tokens x query heads of its group)
// are cut into chunks of up to 64 (48 at 128 dims, 32 at 256), the tokens into splits; a workgroup
// takes one (chunk, split) and its four wavefronts take the 32-token tiles of it in turn, each on
// its own: a wavefront holds its rows' queries and outputs in registers, streams keys and values
// from memory into operand registers in the order in which the cache keeps them, and meets the
// other three only at the end.  No LDS and no barrier lies on the way of a tile.
//
// Per tile, with the 16x16x32 matrix instructions (lane = 16 g + n):
//   S^T = K Q^T: rows are tokens, columns query rows, so lane (n, g) gets the scores of query
//         row n for tokens 16 j + 4 g + i, j < 2, i < 4;
//   O^T = V^T P^T: the same eight tokens are the contraction slots that the lane has to supply
//         of P^T, so the probabilities stay where they are, and the values are stored with the
//         tokens of a block in that order.
// Codes become 16-bit operands exactly: four significant bits, and the block's power of two
// is applied by the conversion relative to a reference exponent (kept so that the products stay
// normal numbers in fp16), whose own power of two sits in the softmax scale (keys) or in
// the unit of the output sums (values).  A change of the values' reference rescales the sums.
//
// Softmax.  One pass with a running maximum m per row, in base 2.  P = 2^(s - m + 8) in fp16: m
// follows a new maximum only once a score passes m + 7 (P would near fp16's largest value), so
// most tiles touch neither the sums nor the other lanes.  Weights down to 2^-22 of the largest
// keep fp16's full 11 bits; their rounding (2^-11 relative) is the only one between the
// stored values and the fp32 sums.  The denominators add the unrounded weights in fp32.  s is
// (sum q k) c; s - m is one multiply-add of the unrounded product, unless m is so large that its
// own rounding (16 at 2^28) would decide the weight: then the product is rounded as m was.
//
// Measured (8 cached heads of 128, bf16): one row and 4 query heads for 64 requests of up to 4096
// tokens 68 us, 5.0 TB/s, bounded by memory; 17 rows for 32 requests of up to 16384 tokens 230 us
// (220 to 237 by the lengths), 480 TFLOP/s, bounded by vector instructions (40% of the time) and the
// matrix unit (27%), which a wavefront uses in turn, and by the longest request; the same of one
// request of 32768 tokens and 8 query heads 39 us.  Chunks of at most 48 rows at 128 dims leave room
// for two wavefronts a SIMD, one of which computes weights while the other multiplies: with one
// wavefront and the compiler's copies of a second set of codes the 17-row call took 540 us.  Three
// row tiles at 128 dims fill the 256 registers of two wavefronts a SIMD and spill three.
//
// Packed rows (kPacked) are the same rows in another place; their splits are equal parts of each request's
// own tiles.  64 single tokens over up to 4096 69 us; 32 drafts of 17 over up to 8192 tokens 142 us.
//
// A NaN among the values reaches only the rows that see its token: a tile that some row does not
// see in full is searched for NaN codes, and where there are any they are taken out of the
// product and put into the visible rows by a second one over indicators.
#include "kv_attention.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

namespace sfx {

namespace {

constexpr int kWaves = 4;
constexpr float kPShift = 8.f;   // P = 2^(s - m + kPShift)
constexpr float kPLimit = 15.f;  // m moves when some s - m + kPShift passes this
constexpr float kNoMax = -3e38f;  // below every score, finite
constexpr float kLarge = 65536.f;  // |m| from which s and m are rounded alike before the difference
constexpr int kRefLo = -5, kRefHi = 7;  // block exponent minus reference: code * 2^that is normal
                                        // in fp16 (2^-9 * 2^-5 = 2^-14, 448 * 2^7 < 65504)

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  using Vec = bf16x8;
  static __device__ Vec widen(unsigned lo, unsigned hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return Vec{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  static __device__ f32x4 mfma(Vec a, Vec b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ unsigned pack(float a, float b) {
    const bf16x2 v{(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(unsigned, v);
  }
};

struct Fp16 {
  using Vec = f16x8;
  static __device__ Vec widen(unsigned lo, unsigned hi, float scale) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true);
    return Vec{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  static __device__ f32x4 mfma(Vec a, Vec b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ unsigned pack(float a, float b) {
    const f16x2 v{(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(unsigned, v);
  }
};

// Three-way maximum of scores as they come from the matrix unit, one instruction (fmaxf would first
// quiet each operand).  A NaN among them stays one: its row is NaN whatever its maximum is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// x y rounded by itself, never as part of a multiply-add.
__device__ __forceinline__ float product(float x, float y) {
#pragma clang fp contract(off)
  float r = x * y;
  asm("" : "+v"(r));
  return r;
}

// Largest / sum over the four lane groups g of a row (lanes n, n + 16, n + 32, n + 48).
__device__ __forceinline__ float group_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What rows [r0, r0 + n) of request b look at: tiles [0, nsink) for the sinks, then
// [first, last).  Tile i of the list is i < nsink ? i : first + i - nsink.
struct Span {
  int start;  // packed: the request's first row, and how many rows it has
  int count;
  int pos0;  // position of the first of the newest tokens
  int rows;  // live rows of the request and head
  int lo_pos, hi_pos;
  int nsink, first, tiles;
};

template <bool kPacked>
__device__ __forceinline__ Span span_of(const KvAttentionArgs& a, int b, int r0, int n) {
  Span s{};
  const int cap = a.max_pages * a.c.page_size;
  int len = a.seq_lens[b], nq;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  if constexpr (kPacked) {
    int from = a.offsets[b], to = a.offsets[b + 1];
    from = from < 0 ? 0 : (from > a.N ? a.N : from);
    to = to < from ? from : (to > a.N ? a.N : to);
    s.start = from;
    s.count = to - from;
    s.pos0 = len - s.count;
    nq = s.count < a.max_q ? s.count : a.max_q;
    if (nq > a.T) nq = 0;  // another call's
  } else {
    nq = a.q_lens ? a.q_lens[b] : a.T;
    nq = nq < 0 ? 0 : (nq > a.T ? a.T : nq);
    s.pos0 = len - nq;
  }
  s.rows = nq * a.group;
  const int r1 = r0 + n < s.rows ? r0 + n : s.rows;
  if (r0 >= r1) return s;
  s.lo_pos = s.pos0 + r0 / a.group;
  s.hi_pos = s.pos0 + (r1 - 1) / a.group;
  const int end = s.hi_pos + 1;
  if (end <= 0) return s;
  const int64_t from = a.window > 0 ? (int64_t)s.lo_pos - a.window + 1 : 0;
  const int lo = from < 0 ? 0 : (int)from;
  s.first = lo / kKvBlock;
  const int sinks = a.sinks < end ? a.sinks : end;
  s.nsink = (sinks + kKvBlock - 1) / kKvBlock;
  s.nsink = s.nsink < s.first ? s.nsink : s.first;
  s.tiles = s.nsink + (end + kKvBlock - 1) / kKvBlock - s.first;
  return s;
}

// Tiles of one split.  Packed calls cut each request's own tiles into equal parts of at least four a
// wavefront; the others cut the table's width.
template <bool kPacked>
__device__ __forceinline__ int per_split(const KvAttentionArgs& a, const Span& s) {
  if constexpr (!kPacked) return a.tiles_per_split;
  const int per = (s.tiles + a.splits - 1) / a.splits;
  return per < 4 * kWaves ? 4 * kWaves : per;
}

// Where the output row of row `row` of request b and head h lies.
template <bool kPacked>
__device__ __forceinline__ int64_t out_row(const KvAttentionArgs& a, const Span& s, int b, int h,
                                           int row) {
  const int64_t token = kPacked ? (int64_t)s.start + row / a.group
                                : (int64_t)b * a.T + row / a.group;
  return token * a.c.heads * a.group + h * a.group + row % a.group;
}

// Zeroes head h's rows of tokens [from, to), every `step`-th.
template <int D>
__device__ void zero_rows(const KvAttentionArgs& a, int h, int64_t from, int64_t to, int64_t step) {
  constexpr int kPieces = D / 8;  // 16-byte pieces of a row
  const int per = a.group * kPieces;
  for (int64_t t = from; t < to; t += step)
    for (int i = threadIdx.x; i < per; i += 64 * kWaves)
      *(u32x4*)((char*)a.out + ((t * a.c.heads + h) * a.group * (int64_t)kPieces + i) * 16) =
          u32x4{0, 0, 0, 0};
}

// Block number of list entry i; its page id (-1: unmapped), read through the scalar cache.
__device__ __forceinline__ int block_of(const Span& s, int i) {
  return __builtin_amdgcn_readfirstlane(i < s.nsink ? i : s.first + i - s.nsink);
}
__device__ __forceinline__ int page_id(const KvAttentionArgs& a, const int32_t* table, int block) {
  return __builtin_amdgcn_readfirstlane(table[kv_page_of(a.c, block)]);
}

// Where a tile lies: its (page, head) and its block there.
struct Place {
  int64_t ph;
  int sub;
  bool mapped;
};
__device__ __forceinline__ Place place_of(const KvAttentionArgs& a, int h, int block, int page) {
  const int per_page = a.c.page_size / kKvBlock;
  const bool mapped = page >= 0 && page < a.c.num_pages;
  return Place{(int64_t)(mapped ? page : 0) * a.c.heads + h,
               block - kv_page_of(a.c, block) * per_page, mapped};
}

template <int D>
__device__ __forceinline__ void load_k(u32x4 (&k)[D / 32], float& scale, const KvAttentionArgs& a,
                                       const Place& p, int off) {
  if (!p.mapped) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) k[c] = u32x4{0, 0, 0, 0};
    scale = 1.f;
    return;
  }
  const uint8_t* base = a.c.k + p.ph * a.c.page_size * D + (int64_t)p.sub * kKvBlock * 64;
#pragma unroll
  for (int tt = 0; tt < 2; ++tt)
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
      k[tt * (D / 64) + j] =
          *(const u32x4*)(base + (int64_t)j * a.c.page_size * 64 + tt * 1024 + off);
  scale = a.c.k_scale[p.ph * (a.c.page_size / kKvBlock) + p.sub];
}

template <int D>
__device__ __forceinline__ void load_v(u32x4 (&v)[D / 32], float& scale, const KvAttentionArgs& a,
                                       const Place& p, int off) {
  if (!p.mapped) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] = u32x4{0, 0, 0, 0};
    scale = 1.f;
    return;
  }
  const uint8_t* base = a.c.v + p.ph * a.c.page_size * D + (int64_t)p.sub * kKvBlock * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) v[c] = *(const u32x4*)(base + c * 1024 + off);
  scale = a.c.v_scale[p.ph * (a.c.page_size / kKvBlock) + p.sub];
}

// Bytes of a dword that are e4m3 NaNs, as 0x80 flags.
__device__ __forceinline__ unsigned nan_bytes(unsigned w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Wavefronts of a SIMD that the registers of a variant leave room for.
constexpr int waves_per_simd(int D, int RT) { return D * RT <= 128 ? 3 : (D * RT <= 384 ? 2 : 1); }

// One (chunk, split): RT 16-row tiles by the split's tokens.
template <typename T, int D, int RT, bool kPacked>
__global__ __launch_bounds__(64 * kWaves, waves_per_simd(D, RT)) void kv_attention_kernel(
    KvAttentionArgs a) {
  constexpr int kSlabs = D / 64, kVc = D / 32;
  constexpr int kPiece = D < 128 ? D : 128;  // dims of one pass of the final reduction
  __shared__ float red[kWaves][16][kPiece + 4];
  __shared__ float sm[kWaves][RT * 16], sl[kWaves][RT * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // a scalar to the compiler
  const int n = lane & 15, g = lane >> 4;

  // Workgroups of one (request, head, split) share its keys and values: their ids are 8 apart, so
  // they run on one XCD and meet in its L2.
  const int per8 = 8 * a.chunks;
  int chunk = (int)(blockIdx.x % per8) / 8;
  // Packed requests have different numbers of chunks.  An XCD deals its workgroups out to its four
  // parts in turn: the chunks' order turns with the group, or all of one chunk would meet in one part
  // (32 drafts of two chunks in a plan of four, beside two chunks of 1024 tokens: 502 us instead of 404
  // for the call).
  if constexpr (kPacked) chunk = (int)((chunk + blockIdx.x / per8) % a.chunks);
  int64_t gi = (int64_t)(blockIdx.x / per8) * 8 + blockIdx.x % 8;
  const int split = (int)(gi % a.splits);
  gi /= a.splits;
  const int h = (int)(gi % a.c.heads);
  const int64_t b64 = gi / a.c.heads;
  if (b64 >= a.B) return;
  const int b = (int)b64;
  const int r0 = chunk * RT * 16, all_rows = a.T * a.group;
  const Span s = span_of<kPacked>(a, b, r0, RT * 16);
  if constexpr (kPacked) {
    if (a.zero && split == 0 && chunk == 0) {
      // rows past max_q, and this request's share of those of no request
      zero_rows<D>(a, h, (int64_t)s.start + a.max_q, (int64_t)s.start + s.count, 1);
      int lo = a.offsets[0], hi = a.offsets[a.B];
      lo = lo < 0 ? 0 : (lo > a.N ? a.N : lo);
      hi = hi < lo ? lo : (hi > a.N ? a.N : hi);
      zero_rows<D>(a, h, b, lo, a.B);
      zero_rows<D>(a, h, (int64_t)hi + b, a.N, a.B);
    }
    if (r0 >= s.rows) return;
  }
  const int per = per_split<kPacked>(a, s);
  const int i0 = split * per;
  if (split > 0 && i0 >= s.tiles) return;
  const int i1 = i0 + per < s.tiles ? i0 + per : s.tiles;
  const int active = (s.tiles + per - 1) / per;

  // queries as the second operand: dims 64 j + 16 g + 8 f + i of row n
  typename T::Vec q[RT][2 * kSlabs];
  int pos[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = r0 + rt * 16 + n;
    const int t = row / a.group;
    const bool live = row < s.rows;
    pos[rt] = live ? s.pos0 + t : -1;
    const int64_t from = kPacked ? ((int64_t)s.start + t) * a.qs.token
                                 : b * a.qs.batch + t * a.qs.token;
    const char* p =
        (const char*)a.q + (from + (h * a.group + row % a.group) * a.qs.head) * 2 + g * 32;
#pragma unroll
    for (int m = 0; m < 2 * kSlabs; ++m) {
      const u32x4 w = live ? (u32x4) * (const u32x4_a2*)(p + (m >> 1) * 128 + (m & 1) * 16)
                           : u32x4{0, 0, 0, 0};
      q[rt][m] = __builtin_bit_cast(typename T::Vec, w);
    }
  }

  f32x4 o[RT][kVc][2];
  float mx[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    mx[rt] = kNoMax;
    l[rt] = 0.f;
#pragma unroll
    for (int c = 0; c < kVc; ++c) o[rt][c][0] = o[rt][c][1] = f32x4{0, 0, 0, 0};
  }
  int kref = 0, vref = 0;
  float cs = a.scale_log2;
  bool first_tile = true, large = false;

  // A tile's codes stay in one set of registers: the next keys are loaded as soon as the scores
  // are made, the next values as soon as the outputs are, each behind the other's work.
  const int32_t* table = a.page_table + (int64_t)b * a.max_pages;
  const int off = n * 64 + g * 16;
  u32x4 kc[kVc], vc[kVc];
  float ks = 1.f, vs = 1.f;
  Place here{};
  int i = i0 + wave, block = 0, next_block = 0, next_page = -1;
  if (i < i1) {
    block = block_of(s, i);
    here = place_of(a, h, block, page_id(a, table, block));
    load_k<D>(kc, ks, a, here, off);
    load_v<D>(vc, vs, a, here, off);
    if (i + kWaves < i1) {
      next_block = block_of(s, i + kWaves);
      next_page = page_id(a, table, next_block);
    }
  }
  for (; i < i1; i += kWaves) {
    const bool more = i + kWaves < i1;
    // reference exponents
    const int ek = __builtin_amdgcn_readfirstlane(kv_exp_of(ks));
    const int ev = __builtin_amdgcn_readfirstlane(kv_exp_of(vs));
    if (first_tile || ek - kref < kRefLo || ek - kref > kRefHi) {
      kref = ek - 1;
      cs = a.scale_log2 * kv_pow2(kref);
    }
    if (first_tile || ev - vref < kRefLo || ev - vref > kRefHi) {
      const float f = kv_pow2(first_tile ? 0 : vref - (ev - 1));
      vref = ev - 1;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < kVc; ++c) {
          o[rt][c][0] *= f;
          o[rt][c][1] *= f;
        }
    }
    first_tile = false;

    // scores
    const float kscale = kv_pow2(ek - kref);
    f32x4 sc[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sc[rt][0] = sc[rt][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < 2 * kSlabs; ++m)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const u32x4 w = kc[tt * kSlabs + (m >> 1)];
        const auto kf = T::widen(w[2 * (m & 1)], w[2 * (m & 1) + 1], kscale);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][tt] = T::mfma(kf, q[rt][m], sc[rt][tt]);
      }
    Place next{};
    if (more) {
      next = place_of(a, h, next_block, next_page);
      load_k<D>(kc, ks, a, next, off);
    }

    // masks: only where some row does not see the whole tile
    const int j0 = block * kKvBlock;
    const bool whole = here.mapped && j0 + kKvBlock - 1 <= s.lo_pos &&
                       (a.window == 0 || s.hi_pos - j0 < a.window || j0 + kKvBlock <= a.sinks);
    if (!whole) {
      unsigned seen[RT];  // bit 4 tt + i: the lane's row sees token 16 tt + 4 g + i
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        seen[rt] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool see = here.mapped && j <= pos[rt] &&
                           (a.window == 0 || pos[rt] - j < a.window || j < a.sinks);
          if (see) seen[rt] |= 1u << e;
          sc[rt][e >> 2][e & 3] = see ? sc[rt][e >> 2][e & 3] : -__builtin_inff();
        }
      }
      unsigned f = 0;
#pragma unroll
      for (int c = 0; c < kVc; ++c)
#pragma unroll
        for (int d = 0; d < 4; ++d) f |= nan_bytes(vc[c][d]);
      if (__any(f != 0)) {
#pragma unroll
        for (int c = 0; c < kVc; ++c)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            // 0x80 flags widened to whole bytes; 0x38 is the code of 1
            const unsigned n0 = (nan_bytes(vc[c][2 * f]) >> 7) * 255u;
            const unsigned n1 = (nan_bytes(vc[c][2 * f + 1]) >> 7) * 255u;
            vc[c][2 * f] &= ~n0;
            vc[c][2 * f + 1] &= ~n1;
            const f16x8 nf = Fp16::widen(n0 & 0x38383838u, n1 & 0x38383838u, 1.f);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              f16x8 see;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                see[e] = (seen[rt] >> e & 1) ? (_Float16)1.f : (_Float16)0.f;
              const f32x4 hit = Fp16::mfma(nf, see, f32x4{0, 0, 0, 0});
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[rt][c][f][e] = hit[e] > 0.f ? __builtin_nanf("") : o[rt][c][f][e];
            }
          }
      }
    }

    // running maximum
    bool move = false;
    float top[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const f32x4 x = sc[rt][0], y = sc[rt][1];
      top[rt] = max3(max3(x[0], x[1], x[2]), max3(x[3], y[0], y[1]), max3(y[2], y[3], y[3]));
      move |= product(top[rt], cs) - mx[rt] > kPLimit - kPShift;
    }
    if (__any(move)) {
      bool wide = false;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float m = fmaxf(mx[rt], product(group_max(top[rt]), cs));
        wide |= fabsf(m) > kLarge && m != kNoMax;
        const float f = __builtin_amdgcn_exp2f(mx[rt] - m);
        mx[rt] = m;
        l[rt] *= f;
#pragma unroll
        for (int c = 0; c < kVc; ++c) {
          o[rt][c][0] *= f;
          o[rt][c][1] *= f;
        }
      }
      large = __any(wide);
    }
    if (large) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sc[rt][e >> 2][e & 3] = product(sc[rt][e >> 2][e & 3], cs) - mx[rt] + kPShift;
    } else {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float bias = kPShift - mx[rt];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sc[rt][e >> 2][e & 3] = fmaf(sc[rt][e >> 2][e & 3], cs, bias);
      }
    }
    f16x8 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = __builtin_amdgcn_exp2f(sc[rt][e >> 2][e & 3]);
        l[rt] += x;
        p[rt][e] = (_Float16)x;
      }
    }

    // outputs
    const float vscale = kv_pow2(ev - vref);
#pragma unroll
    for (int c = 0; c < kVc; ++c)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const f16x8 vf = Fp16::widen(vc[c][2 * f], vc[c][2 * f + 1], vscale);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][c][f] = Fp16::mfma(vf, p[rt], o[rt][c][f]);
      }
    if (more) {
      load_v<D>(vc, vs, a, next, off);
      here = next;
      block = next_block;
      if (i + 2 * kWaves < i1) {
        next_block = block_of(s, i + 2 * kWaves);
        next_page = page_id(a, table, next_block);
      }
    }
  }

  // The four wavefronts' sums, brought to one maximum per row and to the values' own unit.
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = group_sum(l[rt]);
    if (g == 0) {
      sm[wave][rt * 16 + n] = mx[rt];
      sl[wave][rt * 16 + n] = l[rt];
    }
  }
  __syncthreads();
  const float unit = kv_pow2(vref);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float m = sm[0][rt * 16 + n];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sm[w][rt * 16 + n]);
    const float f = __builtin_amdgcn_exp2f(mx[rt] - m) * unit;
#pragma unroll
    for (int c0 = 0; c0 < kVc; c0 += kPiece / 32) {
#pragma unroll
      for (int c = 0; c < kPiece / 32; ++c) {
        f32x4 lo, hi;  // dims 32 c + 8 g + 0..7: element i of half f is dim 2 i + f
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = o[rt][c0 + c][e & 1][e >> 1] * f;
          hi[e] = o[rt][c0 + c][e & 1][2 + (e >> 1)] * f;
        }
        *(f32x4*)&red[wave][n][32 * c + 8 * g] = lo;
        *(f32x4*)&red[wave][n][32 * c + 8 * g + 4] = hi;
      }
      __syncthreads();
      constexpr int kPer = kPiece / 16;  // dims of one thread
      const int rr = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * kPer;
      const int row = r0 + rt * 16 + rr;
      if (row < (kPacked ? s.rows : all_rows)) {
        float mm = sm[0][rt * 16 + rr], ll = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sm[w][rt * 16 + rr]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
          ll += sl[w][rt * 16 + rr] * __builtin_amdgcn_exp2f(sm[w][rt * 16 + rr] - mm);
        float x[kPer];
#pragma unroll
        for (int e = 0; e < kPer; e += 4) {
          f32x4 v = *(const f32x4*)&red[0][rr][d0 + e];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) v += *(const f32x4*)&red[w][rr][d0 + e];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[e + k] = v[k];
        }
        const bool none = ll == 0.f || row >= s.rows;  // sees nothing, or past q_len
        const float inv = 1.f / ll;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = none ? 0.f : x[e] * inv;
        const int d = c0 * 32 + d0;
        if (active > 1) {
          const int64_t rows = (int64_t)a.B * a.c.heads * all_rows;
          const int64_t at = split * rows + ((int64_t)b * a.c.heads + h) * all_rows + row;
#pragma unroll
          for (int e = 0; e < kPer; e += 4)
            *(f32x4*)(a.part_o + at * D + d + e) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
          if (d == 0) a.part_ml[at] = none ? float2{-__builtin_inff(), 0.f} : float2{mm, ll};
        } else {
          const int64_t at = out_row<kPacked>(a, s, b, h, row);
          unsigned* p = (unsigned*)((char*)a.out + (at * D + d) * 2);
#pragma unroll
          for (int e = 0; e < kPer; e += 2) p[e / 2] = T::pack(x[e], x[e + 1]);
        }
      }
      __syncthreads();
    }
  }
}

// Joins the splits of the rows that had more than one: D / 4 lanes hold a row, kGroups such groups
// take every kGroups-th split and meet in LDS.  With many splits one group alone would wait for
// its loads again and again (10 us for 64 splits of 65 rows, 4 with all of a workgroup on a row).
// A split brings its maximum and its sum apart: as one logarithm the sum would be rounded to the
// maximum's step, 4% of a split's weight at scores of 2^20 and all of it at 2^28.
template <typename T, int D, int kGroups, bool kPacked>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttentionArgs a, int chunk_rows) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes / kGroups;
  __shared__ f32x4 xs[kRows][kGroups][kLanes];
  __shared__ float ms[kRows][kGroups], ls[kRows][kGroups];
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes % kGroups;
  const int mine = threadIdx.x / kLanes / kGroups, d = lane * 4;
  const int64_t at = (int64_t)blockIdx.x * kRows + mine;
  const int all_rows = a.T * a.group;
  const int64_t rows = (int64_t)a.B * a.c.heads * all_rows;
  const bool live = at < rows;
  const int row = live ? (int)(at % all_rows) : 0;
  const int h = live ? (int)(at / all_rows % a.c.heads) : 0;
  const int b = live ? (int)(at / all_rows / a.c.heads) : 0;
  const Span s = span_of<kPacked>(a, b, row / chunk_rows * chunk_rows, chunk_rows);
  const int per = per_split<kPacked>(a, s);
  const int active = live && !(kPacked && row >= s.rows) ? (s.tiles + per - 1) / per : 0;
  float m = -__builtin_inff(), l = 0.f;
  f32x4 x{0, 0, 0, 0};
  for (int i = group; active > 1 && i < active; i += 8 * kGroups) {
    float2 ml[8];
    f32x4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = i + k * kGroups < active ? i + k * kGroups : i;
      ml[k] = a.part_ml[j * rows + at];
      o[k] = *(const f32x4*)(a.part_o + (j * rows + at) * D + d);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
    const float z = top == -__builtin_inff() ? 0.f : top;
    const float f = __builtin_amdgcn_exp2f(m - z);
    x *= f;
    l *= f;
    m = top;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k * kGroups < active) {
        // 0 for a split that saw nothing
        const float w = __builtin_amdgcn_exp2f(ml[k].x - z) * ml[k].y;
        l += w;
        x += w * o[k];
      }
  }
  if constexpr (kGroups > 1) {
    xs[mine][group][lane] = x;
    if (lane == 0) {
      ms[mine][group] = m;
      ls[mine][group] = l;
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) m = fmaxf(m, ms[mine][k]);
    const float z = m == -__builtin_inff() ? 0.f : m;
    x = f32x4{0, 0, 0, 0};
    l = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float w = __builtin_amdgcn_exp2f(ms[mine][k] - z);
      l += w * ls[mine][k];
      x += w * xs[mine][k][lane];
    }
  }
  if (active <= 1) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t out = out_row<kPacked>(a, s, b, h, row);
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  *(u32x2*)((char*)a.out + (out * D + d) * 2) =
      u32x2{T::pack(x[0] * inv, x[1] * inv), T::pack(x[2] * inv, x[3] * inv)};
}

// Row tiles of a chunk at most.  At 128 dims a fourth would leave room for one wavefront a SIMD only:
// 64 rows for 32 requests of 8192 tokens took 148 us so and take 124 in two chunks of two.  At 256
// dims two tiles, with one wavefront, take 108 us for 20 rows and 151 for 36 where two chunks of
// one and two wavefronts take 130 and 167.  At 64 dims four against three: 79 us and 91.
int max_row_tiles(int dim) { return dim > 128 ? 2 : (dim > 64 ? 3 : 4); }

// Chunks of equal size: 17 rows of a draft and 4 query heads are five tiles, cut 3 + 3.  Cut 3 + 2
// the smaller chunk runs ahead of the other, the two no longer meet in L2, and the call takes 255 us
// where it takes 237.
int row_tiles(const KvAttentionArgs& a, int dim, int* chunks) {
  const int64_t tiles = ((int64_t)a.T * a.group + 15) / 16;
  const int most = max_row_tiles(dim);
  *chunks = (int)((tiles + most - 1) / most);
  if (*chunks < 1) *chunks = 1;
  return (int)((tiles + *chunks - 1) / *chunks);
}

}  // namespace

size_t kv_attention_plan(KvAttentionArgs* a, int dim) {
  const int rt = row_tiles(*a, dim, &a->chunks);
  const int64_t cap = (int64_t)a->max_pages * a->c.page_size;
  if (a->window >= cap + a->T) a->window = 0;
  int64_t tiles = (cap + kKvBlock - 1) / kKvBlock;
  if (a->window > 0) {
    const int64_t seen = ((int64_t)a->window + a->T) / kKvBlock + 2 +
                         ((int64_t)a->sinks + kKvBlock - 1) / kKvBlock;
    tiles = seen < tiles ? seen : tiles;
  }
  // As many splits as find a place on the card at once (a few more would make a second round of
  // the whole), of at least four tiles a wavefront.
  const int64_t pairs = (int64_t)a->B * a->c.heads * a->chunks;
  const int64_t places = 256 * waves_per_simd(dim, rt);
  int64_t splits = pairs > 0 ? places / pairs : 1;
  const int64_t most = tiles / (4 * kWaves);
  splits = splits > most ? most : splits;
  splits = splits < 1 ? 1 : splits;
  a->tiles_per_split = (int)((tiles + splits - 1) / splits);
  if (a->tiles_per_split < 1) a->tiles_per_split = 1;
  a->splits = (int)splits;
  if (splits == 1) return 0;
  const size_t rows = (size_t)a->B * a->c.heads * a->T * a->group;
  return (size_t)splits * rows * (dim + 2) * sizeof(float);
}

namespace {

// Groups of eight workgroups, one per XCD: see the kernel's decoding of its index.
int64_t grid_of(const KvAttentionArgs& a) {
  return ((int64_t)a.B * a.c.heads * a.splits + 7) / 8 * 8 * a.chunks;
}

}  // namespace

int64_t kv_attention_threads(const KvAttentionArgs& a) {
  return a.B > 0 && a.T > 0 ? grid_of(a) * 64 * kWaves : 0;
}

void kv_attention_place(KvAttentionArgs* a, int dim, void* workspace) {
  const size_t rows = (size_t)a->B * a->c.heads * a->T * a->group;
  a->part_o = (float*)workspace;
  a->part_ml = (float2*)(a->part_o + (size_t)a->splits * rows * dim);
}

namespace {

template <typename T, int D, bool kPacked>
hipError_t launch_rows(const KvAttentionArgs& a, hipStream_t st) {
  int chunks = 0;
  const int rt = row_tiles(a, D, &chunks);
  const dim3 grid((unsigned)grid_of(a));
  const dim3 block(64 * kWaves);
  if (rt == 1)
    hipLaunchKernelGGL((kv_attention_kernel<T, D, 1, kPacked>), grid, block, 0, st, a);
  if (rt == 2)
    hipLaunchKernelGGL((kv_attention_kernel<T, D, 2, kPacked>), grid, block, 0, st, a);
  if constexpr (D <= 128)
    if (rt == 3)
      hipLaunchKernelGGL((kv_attention_kernel<T, D, 3, kPacked>), grid, block, 0, st, a);
  if constexpr (D <= 64)
    if (rt == 4)
      hipLaunchKernelGGL((kv_attention_kernel<T, D, 4, kPacked>), grid, block, 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.B * a.c.heads * a.T * a.group;
  // all of a workgroup on a row where there are many splits (then there are few rows)
  constexpr int kWide = 256 / (D / 4);
  if (a.splits > 4)
    hipLaunchKernelGGL((kv_join_kernel<T, D, kWide, kPacked>), dim3((unsigned)rows), dim3(256), 0,
                       st, a, rt * 16);
  else
    hipLaunchKernelGGL((kv_join_kernel<T, D, 1, kPacked>),
                       dim3((unsigned)((rows * (D / 4) + 255) / 256)), dim3(256), 0, st, a,
                       rt * 16);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_dim(const KvAttentionArgs& a, hipStream_t st) {
  return a.offsets ? launch_rows<T, D, true>(a, st) : launch_rows<T, D, false>(a, st);
}

template <typename T>
hipError_t launch_type(const KvAttentionArgs& a, int dim, hipStream_t st) {
  if (dim == 64) return launch_dim<T, 64>(a, st);
  if (dim == 128) return launch_dim<T, 128>(a, st);
  return launch_dim<T, 256>(a, st);
}

}  // namespace

hipError_t launch_kv_attention(const KvAttentionArgs& a, int dim, KvType type, hipStream_t st) {
  if (a.B <= 0 || a.T <= 0) return hipSuccess;
  return type == kFp16 ? launch_type<Fp16>(a, dim, st) : launch_type<Bf16>(a, dim, st);
}

}  // namespace sfx

// tile_attention.hip -- attention of many rows: whole prompts over their own keys and values, and
// packed chunks over the 8-bit cache.
//
// A request's row t stands at position p (t in a prompt; seq_len - rows + t over the cache) and sees
// the tokens j <= p of its request with, under a window, p - window < j or j < sinks:
//   out_t = sum_j softmax_j(scale q_t . k_j) v_j,    zero for a row that sees nothing.
//
// Decomposition.  The rows of a request and head of keys and values (tokens x query heads of its
// group, the heads of a token next to each other) are cut into tiles of 32 rows a wavefront, 256 a
// workgroup (128 at 256 dims); a workgroup takes one tile by all tokens that its rows see, or by one
// of `splits` equal parts of them where there are few tiles.  Tokens come in tiles of 64 (32 at 256
// dims), brought from memory through registers into one of two LDS buffers while the other is worked
// on: one barrier a tile.  Codes of the cache become 16-bit operands on that way, once for the whole
// workgroup, and their page ids and scales are fetched 64 blocks at a time, one a lane (with scalar
// loads and branches for every tile a chunk of 2048 tokens over 32768 took 1280 us, so 1030).
//
// The loop works on three sets of 32 tokens at once: scores of the next, weights of these, outputs of
// the last.  None waits for another, so the vector instructions of the weights run beside the
// products (8 products of 32 cycles with 48 vector instructions between them take 338 cycles), and
// operands are read from LDS three products ahead.
//
// Per 32 tokens, with the 32x32x16 matrix instructions (lane = 32 h + n):
//   S^T = K Q^T: rows are tokens, columns query rows, so lane (n, h) gets the scores of query
//         row n for the tokens 8 q + 4 h + i, q < 4, i < 4;
//   O^T = V^T P^T: contraction slots may be taken in any order as long as both sides agree, so the
//         lane supplies the probabilities that it has, and V is read in the matching order: rows of
//         four tokens turned by the LDS transposed read (prompts), or eight tokens of a dim in
//         one piece, as the cache has them (chunks, whose keys' rows are permuted to match).
//
// Softmax.  As in kv_attention.hip: one pass, running maximum m per row in base 2,
// P = 2^(s - m + shift), m moves only once a lane's 16 weights of 32 tokens pass 2^(shift + 7) in sum,
// scores past 2^16 are rounded as m is.  P is rounded to the values' type (the matrix unit takes operands
// of one type).  Over the cache and for fp16 prompts that is fp16 with a shift of 8, where weights down to
// 2^-22 of the largest keep 11 bits and the sums of values below 2^16 stay far from fp32's end.  For bf16
// prompts, whose values' range fp16 does not hold, it is bf16, 8 bits, with a shift that follows from
// the number n of 32-token sets: -9 - log2(n), rounded up in log2(n), bounds a row's weights by
// 2 n 2^(shift + 7) <= 1/2, so that no sum of finite values passes fp32's largest, which is bf16's too.
// At the other end products with values below 2^-126 / 2^shift (2^-109 for 8192 tokens) are
// subnormal.  Each weight's rounding is its own, so their error in a sum of many tokens is below the
// result's own rounding.  Denominators add the unrounded weights in fp32.
//
// Infinities and NaN among the values reach only the rows that see their token: they are left out of
// a tile that some row does not see in full, and added at the end to the rows that see them.
//
// Measured (8 heads of keys and values of 128, 4 query heads each, bf16): two prompts of 8192 tokens
// 1045 to 1108 us by the card, 990 to 1050 TFLOP/s, where a library product of 8192^3 reaches 1345; a
// chunk of 2048 tokens over 32768 cached ones 1025 to 1086 us, 920 to 975 TFLOP/s; 16 prompts of 128 to
// 2048 tokens 266 to 294 us by their lengths.  No unit is full: of the cycles the matrix unit is busy in
// 49% (prompts) and 40% (chunks), the LDS in 31% and 27%; of the wavefronts' time a quarter issues vector
// instructions, a quarter to a third waits for loads and barriers and as much for its turn to issue.  The
// clock falls from 2.1 to 1.9 GHz as the matrix unit is kept busier.  At 64 and 256 dims the unit is busy
// in 30% and 28%: half as many products for each weight, and a single wavefront a SIMD, whose waits
// nothing fills.  Workgroups of four wavefronts, two a CU: 1178 us instead of 1055 for the two prompts; a
// higher priority for half the wavefronts: no difference.
#include "tile_attention.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <type_traits>

namespace sfx {

namespace {

constexpr int kDrift = 7;  // P = 2^(s - m + shift); m moves when a lane's weights of 32 tokens pass
                           // 2^(shift + kDrift) in sum
constexpr int kFp16Shift = 8;
constexpr float kNoMax = -3e38f;  // below every score, finite
constexpr float kLarge = 65536.f;  // |m| from which s and m are rounded alike before the difference
constexpr int kRefLo = -5, kRefHi = 7;  // block exponent minus reference: code * 2^that is normal
                                        // in fp16 (2^-9 * 2^-5 = 2^-14, 448 * 2^7 < 65504)

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  static constexpr unsigned kExp = 0x7f80;  // the exponent's bits
  static __device__ float value(unsigned bits) { return __uint_as_float(bits << 16); }
  static __device__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ unsigned pack(float a, float b) {
    const bf16x2 v{(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(unsigned, v);
  }
  template <bool kHi> static __device__ unsigned widen(unsigned codes, float scale) {
    return __builtin_bit_cast(unsigned,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, kHi));
  }
};

struct Fp16 {
  static constexpr unsigned kExp = 0x7c00;
  static __device__ float value(unsigned bits) {
    return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
  }
  static __device__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ unsigned pack(float a, float b) {
    const f16x2 v{(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(unsigned, v);
  }
  template <bool kHi> static __device__ unsigned widen(unsigned codes, float scale) {
    return __builtin_bit_cast(unsigned,
                              __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, kHi));
  }
};

// Three-way maximum of scores as they come from the matrix unit; a NaN among them stays one.
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

// Largest / sum over the two lanes of a row.
__device__ __forceinline__ float pair_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

constexpr int tile_tokens(int D) { return D > 128 ? 32 : 64; }
// Wavefronts of a workgroup.
constexpr int tile_waves(int D) { return D > 128 ? 4 : 8; }
constexpr int tile_rows(int D) { return 32 * tile_waves(D); }

// Segment s of the packed rows: 0 before the first request, 1 .. B the requests, B + 1 behind the
// last.  `edge(s)` is its first token; any memory gives edges within [0, N].
__device__ __forceinline__ int edge(const TileAttentionArgs& a, int s) {
  if (s <= 0) return 0;
  if (s > a.B + 1) return a.N;
  const int o = a.offsets[s - 1];
  return o < 0 ? 0 : (o > a.N ? a.N : o);
}

// A tile of rows, found from its number without a list.  In calls of many requests the tiles of segment
// s are numbers edge(s) * group / rows + s and up, which leaves room for its last, partial one; in
// those of up to 62 they have no gaps.
struct RowTile {
  int seg;                // 0 or B + 1: rows of no request, zeroed
  int start;              // first token of the segment
  int rows, live;         // rows of the segment, those that attend
  int r0;                 // first row of the tile; rows: none
  int pos0;               // position of the segment's first token
  int len;                // tokens of the request
  int lo_pos, hi_pos;     // positions of the tile's rows
  int nsink, first, tiles;  // token tiles: [0, nsink), then [first, ...): `tiles` in all
};

template <int D, bool kPaged>
__device__ __forceinline__ RowTile row_tile(const TileAttentionArgs& a, int vt) {
  constexpr int kRows = tile_rows(D), kTok = tile_tokens(D);
  const int lane = threadIdx.x & 63;
  RowTile t{};
  int end, nth;  // nth: which of the segment's tiles; the last rows see the most tokens and come first
  if (a.B <= 62) {
    // A lane a segment: the running sum of the tiles numbers them without gaps, the rows of no
    // request last.  The workgroups that have work are then the first ones, and where they are just as
    // many as the card has places each finds one (with gaps 16 requests of 512 rows over 8192 tokens,
    // 256 workgroups, took 586 us: some had to wait for others).
    const int seg = lane < a.B ? lane + 1 : (lane == a.B ? 0 : lane);
    const int from = edge(a, seg), to = edge(a, seg + 1);
    int toks = lane < a.B + 2 && to > from ? to - from : 0;
    if constexpr (kPaged)
      if (lane < a.B && a.few > 0 && (toks < a.max_q ? toks : a.max_q) <= a.few) toks = 0;
    const int count = (int)(((int64_t)toks * a.group + kRows - 1) / kRows);
    int sum = count;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(sum, o);
      if (lane >= o) sum += x;
    }
    const uint64_t behind = __ballot(sum > vt);
    if (behind == 0) return t;
    const int at = __builtin_ctzll(behind);
    t.seg = __builtin_amdgcn_readlane(seg, at);
    t.start = __builtin_amdgcn_readlane(from, at);
    end = __builtin_amdgcn_readlane(to, at);
    nth = __builtin_amdgcn_readlane(sum, at) - 1 - vt;
  } else {
    // Largest segment whose first number (see RowTile) is not past vt: 64 probes at a time, the last
    // of neighbours, whose edges are the segment's own.
    int lo = 0, n = a.B + 2, e = 0, hits;
    for (;;) {
      const int step = (n + 63) >> 6, at = lo + lane * step;
      e = edge(a, at);
      const bool ok = lane * step < n && (int64_t)e * a.group / kRows + at <= vt;
      hits = 64 - __builtin_clzll(__ballot(ok) | 1);
      if (step == 1) break;
      lo += (hits - 1) * step;
      const int left = n - (hits - 1) * step;
      n = left < step ? left : step;
    }
    t.seg = __builtin_amdgcn_readfirstlane(lo + hits - 1);
    t.start = __builtin_amdgcn_readlane(e, hits - 1);
    end = hits < 64 ? __builtin_amdgcn_readlane(e, hits & 63)
                    : __builtin_amdgcn_readfirstlane(edge(a, t.seg + 1));
    const int count =
        end > t.start ? (int)(((int64_t)(end - t.start) * a.group + kRows - 1) / kRows) : 0;
    nth = count - 1 - (vt - (int)((int64_t)t.start * a.group / kRows) - t.seg);
  }
  const int toks = end > t.start ? end - t.start : 0;
  t.rows = toks * a.group;
  t.r0 = nth >= 0 ? nth * kRows : t.rows;
  if (t.seg == 0 || t.seg == a.B + 1) return t;
  t.live = t.rows;
  t.len = toks;
  if constexpr (kPaged) {
    const int b = t.seg - 1, cap = a.max_pages * a.c.page_size;
    const int len = __builtin_amdgcn_readfirstlane(a.seq_lens[b]);
    t.len = len < 0 ? 0 : (len > cap ? cap : len);
    t.pos0 = t.len - toks;
    const int attend = toks < a.max_q ? toks : a.max_q;
    t.live = attend * a.group;
    if (a.few > 0 && attend <= a.few) {
      t.r0 = t.rows;
      return t;
    }
  }
  const int r1 = t.r0 + kRows < t.live ? t.r0 + kRows : t.live;
  if (t.r0 >= r1) return t;
  t.lo_pos = t.pos0 + t.r0 / a.group;
  t.hi_pos = t.pos0 + (r1 - 1) / a.group;
  const int upto = t.hi_pos + 1;
  if (upto <= 0) return t;
  const int64_t from = a.window > 0 ? (int64_t)t.lo_pos - a.window + 1 : 0;
  t.first = (from < 0 ? 0 : (int)from) / kTok;
  const int sinks = a.sinks < upto ? a.sinks : upto;
  t.nsink = (sinks + kTok - 1) / kTok;
  t.nsink = t.nsink < t.first ? t.nsink : t.first;
  t.tiles = t.nsink + (upto + kTok - 1) / kTok - t.first;
  return t;
}

// Token tiles of one split.
__device__ __forceinline__ int per_split(const TileAttentionArgs& a, const RowTile& t) {
  const int per = (t.tiles + a.splits - 1) / a.splits;
  return per < a.least ? a.least : per;
}

// Bytes of a dword that are e4m3 NaNs, as 0x80 flags.
__device__ __forceinline__ unsigned nan_bytes(unsigned w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Where the head's output row of row r of a segment lies.
__device__ __forceinline__ int64_t out_row(const TileAttentionArgs& a, const RowTile& t, int h,
                                           int r) {
  return ((int64_t)t.start + r / a.group) * a.heads * a.group + h * a.group + r % a.group;
}

// Page id of a block of 32 cached tokens; -1 where it is unmapped or past the table.  (Calls without any
// pages have no tokens.)  Unmapped blocks are read as page 0's and not seen.
__device__ __forceinline__ int page_of(const TileAttentionArgs& a, const int32_t* table, int block) {
  const int pi = kv_page_of(a.c, block), last = a.max_pages - 1;
  const int id = table[pi < last ? pi : last];
  return pi > last || (unsigned)id >= (unsigned)a.c.num_pages ? -1 : id;
}

// One (tile of rows, head, split).
template <typename T, int D, bool kPaged>
__global__ __launch_bounds__(64 * tile_waves(D), tile_waves(D) / 4) void tile_attention_kernel(
    TileAttentionArgs a) {
  using P = std::conditional_t<kPaged, Fp16, T>;  // type of probabilities and values
  constexpr int kThreads = 64 * tile_waves(D);
  constexpr int kTok = tile_tokens(D), kHalves = kTok / 32;
  constexpr int kPieces = kTok * D / 8;  // 16-byte pieces of a tile in LDS
  constexpr int kLoads = kPaged ? (kPieces / 2 + kThreads - 1) / kThreads : kPieces / kThreads;
  constexpr int kDimTiles = D / 32, kSteps = D / 16;
  // of two 16-bit values: their exponents, and what carries exponents of all ones into the signs
  constexpr unsigned kExps = P::kExp * 0x10001u, kCarry = (0x8000u - P::kExp) * 0x10001u;
  // LDS: keys by token, values by token (prompts) or by block and dim, four groups of eight tokens
  // each (chunks).  The rows' padding spreads what a wavefront reads at once over all banks: 16 rows
  // at one 16-byte piece, or 4 tokens by 64 bytes.
  constexpr int kKeyRow = 2 * D + 16, kKeyHalf = 32 * kKeyRow;
  constexpr int kValueRow = kPaged ? 80 : 2 * D + 64;
  constexpr int kValueHalf = (kPaged ? D : 32) * kValueRow;
  constexpr int kValueSlots = kHalves > 1 ? 2 : 3;
  __shared__ __attribute__((aligned(16))) char lds_k[2][kHalves * kKeyHalf];
  __shared__ __attribute__((aligned(16))) char lds_v[kValueSlots][kHalves * kValueHalf];
  __shared__ int special;

  // Workgroups that follow each other go to different XCDs; a head's stay on the same ones.
  const int h = blockIdx.x % a.heads;
  const unsigned rest = blockIdx.x / a.heads;
  const int split = rest % a.splits;
  const RowTile t = row_tile<D, kPaged>(a, rest / a.splits);
  if (t.r0 >= t.rows) return;
  const int per = per_split(a, t);
  const int i0 = split * per;
  if (split > 0 && i0 >= t.tiles) return;
  const int i1 = i0 + per < t.tiles ? i0 + per : t.tiles;
  const int active = (t.tiles + per - 1) / per;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, hh = lane >> 5;
  const int w0 = t.r0 + wave * 32;  // the wavefront's rows
  const int row = w0 + n;
  const bool live = row < t.live;
  const int pos = live ? t.pos0 + row / a.group : -1;
  // positions of the wavefront's rows; lo > hi: none
  const int w1 = w0 + 32 < t.live ? w0 + 32 : t.live;
  const int lo_pos = w0 < t.live ? t.pos0 + w0 / a.group : 0;
  const int hi_pos = w0 < t.live ? t.pos0 + (w1 - 1) / a.group : -1;

  // queries as the second operand: dims 16 m + 8 hh + i of row n
  u32x4 q[kSteps];
  {
    const int64_t at = ((int64_t)t.start + row / a.group) * a.qs.token +
                       (int64_t)(h * a.group + row % a.group) * a.qs.head;
    const char* p = (const char*)a.q + at * 2 + hh * 16;
#pragma unroll
    for (int m = 0; m < kSteps; ++m)
      q[m] = live ? (u32x4) * (const u32x4_a2*)(p + m * 32) : u32x4{0, 0, 0, 0};
  }

  f32x16 o[kDimTiles];
#pragma unroll
  for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[c][e] = 0.f;
  float mx = kNoMax, l = 0.f;
  bool large = false;      // scores are rounded as the maximum is
  // weights' power of two, see the head: of bf16 such that all weights of a row stay below 1/2 in sum
  const int sets = t.tiles * kHalves;
  const int shift_log2 = std::is_same_v<P, Fp16>
                             ? kFp16Shift
                             : -(kDrift + 2 + (sets > 1 ? 32 - __builtin_clz(sets - 1) : 0));
  const float shift = (float)shift_log2, sum_limit = kv_pow2(shift_log2 + kDrift);
  float limit = sum_limit;  // of a lane's weights of 32 tokens; with large scores any is too much

  // ---- tokens on their way: a tile's pieces in registers.  Keys are a tile ahead of the values.
  u32x4 kr[kLoads], vr[kLoads];
  const int32_t* table = kPaged ? a.page_table + (int64_t)(t.seg - 1) * a.max_pages : nullptr;
  auto first_block = [&](int i) {  // 32-token block of list entry i
    return __builtin_amdgcn_readfirstlane((i < t.nsink ? i : t.first + i - t.nsink) * kHalves);
  };
  // Of cached tokens: what is known of 64 blocks, one a lane, in the order of the list, and of the 64
  // after them.  Pages are asked for a batch ahead and scales half a batch, so that a tile takes what
  // it needs from the lanes and waits for nothing.
  int pages = -1, packed = 0;    // packed: exponents + 64 of keys and values, place in the page
  int pages_next = -1, sub_next = 0;
  float ks_next = 1.f, vs_next = 1.f;
  const int per_page = a.c.page_size / kKvBlock;
  auto ask_pages = [&](int q) {  // q: list position of the batch's first block, from i0 on
    int i = i0 + (q + lane) / kHalves;
    i = i < i1 ? i : i1 - 1;
    const int block = (i < t.nsink ? i : t.first + i - t.nsink) * kHalves + (q + lane) % kHalves;
    pages_next = page_of(a, table, block);
    sub_next = block - kv_page_of(a.c, block) * per_page;
  };
  auto ask_scales = [&]() {
    const int64_t at = ((int64_t)(pages_next < 0 ? 0 : pages_next) * a.c.heads + h) * per_page + sub_next;
    ks_next = a.c.k_scale[at];
    vs_next = a.c.v_scale[at];
  };
  auto take_batch = [&]() {
    pages = pages_next;
    packed = (kv_exp_of(ks_next) + 64) | (kv_exp_of(vs_next) + 64) << 8 | sub_next << 16;
  };
  // Of a tile, as its keys are loaded: its blocks' pages and the rest.
  struct Info {
    int page[kHalves], packed[kHalves];
    int vref[kHalves];  // the unit in which the values lie in LDS
  };
  Info now{}, next{}, before{};  // of the tile whose weights are made, the one behind it, the last
  int ref = 0;                   // the values' reference exponent, in the order of their tiles
  float vscale[kHalves];
  bool any_ref = false;
  // a thread's pieces of a tile of 16-bit tokens
  auto load_rows = [&](u32x4(&r)[kLoads], const void* from, const KvStrides& s, int i) {
    const int j0 = first_block(i) * 32, last = t.len - 1 - j0;
    const char* p = (const char*)from + (((int64_t)t.start + j0) * s.token + h * s.head) * 2;
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = threadIdx.x + y * kThreads, off = c % (D / 8) * 16, tok = c / (D / 8);
      const unsigned u = tok < last ? tok : last;  // those past the end are seen by no row
      r[y] = *(const u32x4_a2*)(p + u * (uint64_t)(s.token * 2) + off);
    }
  };
  // a thread's pieces of a tile of codes: 16 codes each, of block c / 2D
  auto piece = [&](int y) {
    const int c = threadIdx.x + y * kThreads;
    return kPieces / 2 % kThreads ? c % (kPieces / 2) : c;  // too many threads load twice
  };
  const int64_t page_bytes = (int64_t)a.c.heads * a.c.page_size * D;
  const int64_t head_bytes = (int64_t)h * a.c.page_size * D;
  auto load_codes = [&](u32x4(&r)[kLoads], const uint8_t* codes, const Info& f, bool val) {
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int x = kHalves > 1 ? __builtin_amdgcn_readfirstlane(piece(y) / (2 * D)) : 0;
      const int page = x ? f.page[kHalves - 1] : f.page[0];
      const int sub = (x ? f.packed[kHalves - 1] : f.packed[0]) >> 16;
      const uint8_t* p = codes + head_bytes + (page < 0 ? 0 : page) * page_bytes +
                         sub * (kKvBlock * (val ? D : 64));
      // keys: slab u / 128, token u / 4 of it, dims 16 (u % 4) and up
      const unsigned u = piece(y) % (2 * D);
      r[y] = *(const u32x4*)(p + (val ? u * 16 : (u >> 7) * (a.c.page_size * 64u) + (u & 127) * 16));
    }
  };
  auto load_k = [&](Info& f, int i) {
    if constexpr (kPaged) {
      const int q = (i - i0) * kHalves;
      if ((q & 63) == 0) {
        take_batch();
        ask_pages(q + 64);
      } else if ((q & 63) == 32) {
        ask_scales();
      }
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        f.page[x] = __builtin_amdgcn_readlane(pages, (q & 63) + x);
        f.packed[x] = __builtin_amdgcn_readlane(packed, (q & 63) + x);
      }
      load_codes(kr, a.c.k, f, false);
    } else {
      load_rows(kr, a.k, a.ks, i);
    }
  };
  auto load_v = [&](Info& f, int i) {
    if constexpr (kPaged)
      load_codes(vr, a.c.v, f, true);
    else
      load_rows(vr, a.v, a.vs, i);
  };
  // Registers to LDS.
  auto store_k = [&](char* kl) {
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = threadIdx.x + y * kThreads;
      if constexpr (kPaged) {
        if (kPieces / 2 % kThreads && c >= kPieces / 2) continue;
        const int x = __builtin_amdgcn_readfirstlane(c / (2 * D)), u = c % (2 * D);
        // token 16 j + 8 s + 4 h + i goes to row 16 s + 8 j + 4 h + i
        const int tok = (u & 127) >> 2, r = (tok & 7) | (tok & 8) << 1 | (tok & 16) >> 1;
        const int at = x * 32 + r, piece = (u >> 7) * 8 + (u & 3) * 2;
        u32x4 w[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e >> 1][2 * (e & 1)] = T::template widen<false>(kr[y][e], 1.f);
          w[e >> 1][2 * (e & 1) + 1] = T::template widen<true>(kr[y][e], 1.f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *(u32x4*)(kl + at * kKeyRow + (piece + e) * 16) = w[e];
      } else {
        const int tok = c / (D / 8), piece = c % (D / 8);
        *(u32x4*)(kl + tok * kKeyRow + piece * 16) = kr[y];
      }
    }
  };
  // Of a tile that some row does not see in full the infinities and NaN among the values are left
  // out (0 times one would be NaN in every row) and dealt with at the end.
  auto store_v = [&](char* vl, Info& f, bool clean) {
    if constexpr (kPaged)
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        const int ev = (f.packed[x] >> 8 & 255) - 64;
        if (!any_ref || ev - ref < kRefLo || ev - ref > kRefHi) ref = ev - 1;
        any_ref = true;
        f.vref[x] = ref;
        vscale[x] = kv_pow2(ev - ref);
      }
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = threadIdx.x + y * kThreads;
      if constexpr (kPaged) {
        if (kPieces / 2 % kThreads && c >= kPieces / 2) continue;
        const int x = __builtin_amdgcn_readfirstlane(c / (2 * D)), u = c % (2 * D);
        // [block][dim][4 groups of eight tokens]
        const int dim = (u >> 6) * 32 + (u >> 2 & 15) * 2, g = u & 3;
        const float sc = vscale[kHalves > 1 && x ? kHalves - 1 : 0];
        if (clean) {
          unsigned bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned nan = nan_bytes(vr[y][e]);
            bad |= nan;
            vr[y][e] &= ~((nan >> 7) * 255u);
          }
          if (__any(bad != 0)) special = 1;
        }
        u32x4 w[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e >> 1][2 * (e & 1)] = Fp16::widen<false>(vr[y][e], sc);
          w[e >> 1][2 * (e & 1) + 1] = Fp16::widen<true>(vr[y][e], sc);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
          *(u32x4*)(vl + (x * D + dim + f) * kValueRow + g * 16) = w[f];
      } else {
        const int tok = c / (D / 8), piece = c % (D / 8);
        if (clean) {
          unsigned bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned f = ((vr[y][e] & kExps) + kCarry) & 0x80008000u;
            bad |= f;
            vr[y][e] &= ~((f >> 15) * 0xffffu);
          }
          if (__any(bad != 0)) special = 1;
        }
        *(u32x4*)(vl + tok * kValueRow + piece * 16) = vr[y];
      }
    }
  };

  // ---- operands of 32 tokens from LDS
  auto key = [&](const char* kl, int m) {
    return *(const u32x4*)(kl + n * kKeyRow + hh * 16 + m * 32);
  };
  // number g: of step g / kDimTiles (16 slots) and dims 32 (g % kDimTiles): [lane's dim][its tokens]
  auto value = [&](const char* vl, int g) {
    const int s = g / kDimTiles, c = g % kDimTiles;
    if constexpr (kPaged) {
      return *(const u32x4*)(vl + n * kValueRow + hh * 16 + s * 32 + c * 32 * kValueRow);
    } else {
      const char* p = vl + (4 * hh + (lane >> 2 & 3)) * kValueRow + (lane >> 4 & 1) * 32 +
                      (lane & 3) * 8 + s * 16 * kValueRow + c * 64;
      u32x4 r;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u32x2 w = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                       (__attribute__((address_space(3))) i16x4*)(char*)(p + x * 8 * kValueRow)));
        r[2 * x] = w[0];
        r[2 * x + 1] = w[1];
      }
      return r;
    }
  };
  // token of score e of a half
  auto token = [&](int e) {
    return kPaged ? 16 * (e >> 2 & 1) + 8 * (e >> 3) + 4 * hh + (e & 3)
                  : 8 * (e >> 2) + 4 * hh + (e & 3);
  };

  auto sees = [&](int j, int pos) {
    return j <= pos && (a.window == 0 || pos - j < a.window || j < a.sinks);
  };
  // every row of the workgroup sees the whole tile
  auto all_see = [&](int j0) {
    return j0 + kTok - 1 <= t.lo_pos &&
           (a.window == 0 || t.hi_pos - j0 < a.window || j0 + kTok <= a.sinks);
  };

  if (threadIdx.x == 0) special = 0;
  __syncthreads();
  int unit = 0;  // the output sums' power of two

  // ---- work on 32 tokens.  Operands are read kAhead steps before they are used.
  constexpr int kAhead = 3;
  u32x4 kf[kAhead + 1], vf[kAhead + 1];
  struct Weights {
    u32x4 w[2];
  };
  auto read_ahead = [&](const char* kl, const char* vl) {
#pragma unroll
    for (int g = 0; g < kAhead; ++g) {
      kf[g] = key(kl, g);
      vf[g] = value(vl, g);
    }
  };
  // In one go, so that the matrix unit waits for nothing: scores of the 32 tokens behind (keys kl),
  // outputs of the 32 before (values vl, weights pb), and the weights pc of these, against the running
  // maximum as it is.  No weight passes the limit unless their sum does, so the sum tells whether the
  // maximum has to move.  kl2, vl2: whose operands are read ahead at the end (NULL: none).
  auto step = [&](const char* kl, const char* vl, const f32x16& s, f32x16& sn, const Weights& pb,
                  Weights& pc, float cs, const char* kl2, const char* vl2) {
    const float bias = shift - mx;
    float add[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 16; ++e) sn[e] = 0.f;
#pragma unroll
    for (int g = 0; g < kSteps; ++g) {
      constexpr int kRing = kAhead + 1;
      const int ga = g + kAhead;
      if (ga < kSteps) {
        kf[ga % kRing] = key(kl, ga);
        vf[ga % kRing] = value(vl, ga);
      } else if (kl2) {
        kf[ga % kRing] = key(kl2, ga - kSteps);
        vf[ga % kRing] = value(vl2, ga - kSteps);
      }
      sn = T::mfma(kf[g % kRing], q[g], sn);
      o[g % kDimTiles] = P::mfma(vf[g % kRing], pb.w[g / kDimTiles], o[g % kDimTiles]);
      // two weights or more at a time: every second step's where there are more steps than pairs
      constexpr int kPairs = kSteps < 8 ? kSteps : 8;
      if (g % (kSteps / kPairs) == 0)
#pragma unroll
        for (int e = 16 / kPairs * (g * kPairs / kSteps); e < 16 / kPairs * (g * kPairs / kSteps + 1);
             e += 2) {
          const float u = __builtin_amdgcn_exp2f(fmaf(s[e], cs, bias));
          const float v = __builtin_amdgcn_exp2f(fmaf(s[e + 1], cs, bias));
          add[0] += u;
          add[1] += v;
          unsigned w = P::pack(u, v);
          // made here, not where it is needed
          asm volatile("" : "+v"(w), "+v"(add[0]), "+v"(add[1]));
          pc.w[e >> 3][(e & 7) >> 1] = w;
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    return add[0] + add[1];
  };
  // The same with the maximum brought up to date; scores that are large are rounded as it is.
  auto weights_moved = [&](const f32x16& s, float cs, float& sum) {
    float top = max3(s[0], s[1], s[2]);
#pragma unroll
    for (int e = 3; e < 15; e += 2) top = max3(top, s[e], s[e + 1]);
    top = product(max3(top, s[15], s[15]), cs);
    if (__any(top - mx > 0.f)) {
      const float m = fmaxf(mx, pair_max(top));
      large = __any(fabsf(m) > kLarge && m != kNoMax);
      limit = large ? -1.f : sum_limit;
      const float f = __builtin_amdgcn_exp2f(mx - m);
      mx = m;
      l *= f;
#pragma unroll
      for (int c = 0; c < kDimTiles; ++c) o[c] *= f;
    }
    Weights r;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float u[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u[k] = large ? product(s[e + k], cs) - mx + shift : fmaf(s[e + k], cs, shift - mx);
        u[k] = __builtin_amdgcn_exp2f(u[k]);
        sum += u[k];
      }
      r.w[e >> 3][(e & 7) >> 1] = P::pack(u[0], u[1]);
    }
    return r;
  };
  auto to_unit = [&](int to) {
    if (kPaged && to != unit) {
      const float f = kv_pow2(unit - to);
      unit = to;
#pragma unroll
      for (int c = 0; c < kDimTiles; ++c) o[c] *= f;
    }
  };

  // ---- the loop
  int ks = 0, vs = 0;  // tile i's slots
  auto turn = [&](int s, int n) { return s + 1 == n ? 0 : s + 1; };
  if (i0 < i1) {
    if constexpr (kPaged) {
      ask_pages(0);
      ask_scales();
    }
    load_k(now, i0);
    load_v(now, i0);
    store_k(lds_k[0]);
    if (i0 + 1 < i1) load_k(next, i0 + 1);
    // what the first outputs are made of: nothing
    for (int c = threadIdx.x; c < kValueHalf / 16; c += kThreads)
      *(u32x4*)(lds_v[kValueSlots - 1] + (kHalves - 1) * kValueHalf + c * 16) = u32x4{0, 0, 0, 0};
  }
  // Tile i's values and tile i + 1's keys to LDS, those behind them on their way.  The slots are not
  // read by wavefronts that are still in the last round: they are past its barrier.
  auto bring = [&](int i, Info& after) {
    bool clean = !all_see(first_block(i) * 32);
    if constexpr (kPaged)
#pragma unroll
      for (int x = 0; x < kHalves; ++x) clean |= now.page[x] < 0;
    store_v(lds_v[vs], now, clean);
    if (i + 1 < i1) {
      store_k(lds_k[ks ^ 1]);
      load_v(next, i + 1);
      if (i + 2 < i1) load_k(after, i + 2);
    }
  };
  __syncthreads();
  // the wavefront's own tiles end earlier than the workgroup's
  int iw = i1;
  while (iw > i0 && first_block(iw - 1) * 32 > hi_pos) --iw;
  f32x16 sc[2];  // of this half and the next
  Weights p[2];  // of the last half and this
#pragma unroll
  for (int e = 0; e < 16; ++e) sc[0][e] = 0.f;
#pragma unroll
  for (int m = 0; m < kSteps; ++m) sc[0] = T::mfma(key(lds_k[0], m), q[m], sc[0]);
  p[1].w[0] = p[1].w[1] = u32x4{0, 0, 0, 0};
  if constexpr (kHalves > 1)
    read_ahead(lds_k[0] + kKeyHalf, lds_v[kValueSlots - 1] + kValueHalf);
  for (int i = i0; i < iw; ++i) {
    const int j0 = first_block(i) * 32;
    const char *k_now = lds_k[ks], *k_next = lds_k[ks ^ 1], *v_now = lds_v[vs];
    const char* v_last = lds_v[vs == 0 ? kValueSlots - 1 : vs - 1];
    Info after{};
    bring(i, after);
#pragma unroll
    for (int x = 0; x < kHalves; ++x) {
      const int jx = j0 + 32 * x;
      const float cs = kPaged ? a.scale_log2 * kv_pow2((now.packed[x] & 255) - 64) : a.scale_log2;
      f32x16& s = sc[kHalves > 1 ? x : 0];
      f32x16& sn = sc[kHalves > 1 ? 1 - x : 1];
      Weights& pb = p[kHalves > 1 ? 1 - x : 1];
      Weights& pc = p[kHalves > 1 ? x : 0];
      if (x == kHalves - 1) {
        __syncthreads();
        read_ahead(k_next, kHalves > 1 ? v_now : v_last);
      }
      to_unit(x > 0 ? now.vref[x > 0 ? x - 1 : 0] : before.vref[kHalves - 1]);
      const bool mapped = !kPaged || now.page[x] >= 0;
      const bool whole = mapped && jx + 31 <= lo_pos &&
                         (a.window == 0 || hi_pos - jx < a.window || jx + 32 <= a.sinks);
      if (!whole) {
        int at = pos;
        asm("" : "+v"(at));  // keeps what follows out of the other path's registers
#pragma unroll
        for (int e = 0; e < 16; ++e)
          s[e] = mapped && sees(jx + token(e), at) ? s[e] : -__builtin_inff();
      }
      float sum;
      if constexpr (kHalves == 1)
        sum = step(k_next, v_last, s, sn, pb, pc, cs, nullptr, nullptr);
      else if (x == 0)
        sum = step(k_now + kKeyHalf, v_last + kValueHalf, s, sn, pb, pc, cs, nullptr, nullptr);
      else
        sum = step(k_next, v_now, s, sn, pb, pc, cs, k_next + kKeyHalf, v_now + kValueHalf);
      if (__any(sum > limit)) pc = weights_moved(s, cs, sum);
      l += sum;
      if constexpr (kHalves == 1) {
        s = sn;
        pb = pc;
      }
    }
    ks ^= 1;
    vs = turn(vs, kValueSlots);
    before = now;
    now = next;
    next = after;
  }
  if (i0 < iw) {  // the last outputs
    to_unit(before.vref[kHalves - 1]);
    const char* vl = lds_v[vs == 0 ? kValueSlots - 1 : vs - 1] + (kHalves - 1) * kValueHalf;
#pragma unroll
    for (int g = 0; g < kSteps; ++g)
      o[g % kDimTiles] = P::mfma(value(vl, g), p[1].w[g / kDimTiles], o[g % kDimTiles]);
  }
  for (int i = iw; i < i1; ++i) {  // for the others
    Info after{};
    bring(i, after);
    __syncthreads();
    ks ^= 1;
    vs = turn(vs, kValueSlots);
    now = next;
    next = after;
  }

  // Infinities and NaN that `store` took out: added to the rows that see their tokens.
  __syncthreads();
  if (special) {
    for (int i = i0; i < i1; ++i) {
      const int j0 = first_block(i) * 32;
      bool left_out = !all_see(j0);
      if constexpr (kPaged)
#pragma unroll
        for (int x = 0; x < kHalves; ++x)
          left_out |= __builtin_amdgcn_readfirstlane(page_of(a, table, j0 / 32 + x)) < 0;
      if (!left_out) continue;
#pragma unroll 1
      for (int u = 0; u < kTok; ++u) {
        const int j = j0 + u;
        if (j >= t.len || !__any(sees(j, pos))) continue;
        const bool see = sees(j, pos);
        if constexpr (kPaged) {
          const int block = __builtin_amdgcn_readfirstlane(j >> 5);
          const int page = __builtin_amdgcn_readfirstlane(page_of(a, table, block));
          if (page < 0) continue;
          const int sub = block - kv_page_of(a.c, block) * per_page;
          const uint8_t* p = a.c.v + head_bytes + page * page_bytes + sub * (kKvBlock * D) +
                             (u >> 2 & 3) * 16 + (u >> 4 & 1) * 4 + (u & 3);
#pragma unroll
          for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int dim = 8 * (e >> 2) + 4 * hh + (e & 3);
              if (see && (p[c * 1024 + (dim >> 1) * 64 + (dim & 1) * 8] & 127) == 127)
                o[c][e] = __builtin_nanf("");
            }
        } else {
          const unsigned short* p = (const unsigned short*)a.v +
                                    (((int64_t)t.start + j) * a.vs.token + h * a.vs.head);
#pragma unroll
          for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const unsigned v = p[32 * c + 8 * (e >> 2) + 4 * hh + (e & 3)];
              if (see && (v & P::kExp) == P::kExp) o[c][e] += P::value(v);
            }
        }
      }
    }
  }

  // results: lane (n, hh) holds row n, dims 32 c + 8 q + 4 hh + i
  l = pair_sum(l);
  const bool none = l == 0.f || !live;
  const float f = none ? 0.f : kv_pow2(unit) / l;
#pragma unroll
  for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[c][e] = none ? 0.f : o[c][e] * f;
  if (active > 1) {
    const int64_t rows = (int64_t)a.N * a.heads * a.group;
    const int64_t at = split * rows + out_row(a, t, h, row);
    if (row < t.rows) {
#pragma unroll
      for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(f32x4*)(a.part_o + at * D + 32 * c + 8 * g + 4 * hh) =
              f32x4{o[c][4 * g], o[c][4 * g + 1], o[c][4 * g + 2], o[c][4 * g + 3]};
      if (hh == 0) a.part_ml[at] = none ? float2{-__builtin_inff(), 0.f} : float2{mx, l};
    }
    return;
  }
  char* to = (char*)a.out + out_row(a, t, h, row) * (2 * D);
#pragma unroll
  for (int c = 0; c < kDimTiles; ++c)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      // the two lanes of a row exchange halves: 16 bytes each
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned x = T::pack(o[c][4 * g + 2 * e], o[c][4 * g + 2 * e + 1]);
        const unsigned y = T::pack(o[c][4 * g + 4 + 2 * e], o[c][4 * g + 5 + 2 * e]);
        const auto z = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        w[e] = z[0];
        w[2 + e] = z[1];
      }
      if (row < t.rows) *(u32x4*)(to + (32 * c + 8 * g + 8 * hh) * 2) = w;
    }
}

// Joins the splits of the tiles that had more than one, in order: D / 4 lanes a row.
template <typename T, int D, bool kPaged>
__global__ __launch_bounds__(256) void tile_join_kernel(TileAttentionArgs a) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes, kParts = tile_rows(D) / kRows;
  const int part = blockIdx.x % kParts;
  const unsigned rest = blockIdx.x / kParts;
  const int h = rest % a.heads;
  const RowTile t = row_tile<D, kPaged>(a, rest / a.heads);
  const int per = per_split(a, t);
  const int active = (t.tiles + per - 1) / per;
  const int row = t.r0 + part * kRows + threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  if (active <= 1 || row >= t.rows) return;
  const int64_t rows = (int64_t)a.N * a.heads * a.group, at = out_row(a, t, h, row);
  float m = -__builtin_inff(), l = 0.f;
  f32x4 x{0, 0, 0, 0};
  for (int i = 0; i < active; i += 8) {
    float2 ml[8];
    f32x4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = i + k < active ? i + k : i;
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
      if (i + k < active) {
        // 0 for a split that saw nothing
        const float w = __builtin_amdgcn_exp2f(ml[k].x - z) * ml[k].y;
        l += w;
        x += w * o[k];
      }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(u32x2*)((char*)a.out + (at * D + d) * 2) =
      u32x2{T::pack(x[0] * inv, x[1] * inv), T::pack(x[2] * inv, x[3] * inv)};
}

// Numbers of row tiles (see RowTile).
int64_t tile_numbers(const TileAttentionArgs& a, int dim) {
  return (int64_t)a.N * a.group / tile_rows(dim) + a.B + 2;
}

}  // namespace

size_t tile_attention_plan(TileAttentionArgs* a, int dim, bool paged) {
  const int64_t cap = paged ? (int64_t)a->max_pages * a->c.page_size : a->N;
  if (a->window >= cap + a->N) a->window = 0;
  const int tok = tile_tokens(dim);
  int64_t tiles = (cap + tok - 1) / tok;
  if (a->window > 0) {
    const int64_t seen = ((int64_t)a->window + tile_rows(dim) / a->group) / tok + 2 +
                         ((int64_t)a->sinks + tok - 1) / tok;
    tiles = seen < tiles ? seen : tiles;
  }
  // As many splits as find a place on the card at once, of at least four tiles.
  a->least = 4;
  int64_t row_tiles = (int64_t)a->N * a->group / tile_rows(dim);
  // Every request has one.  Where those of few rows are left out their rows count all the same, as the
  // plan does not know the offsets: many drafts beside one short chunk leave it with too few splits.
  const int64_t least = a->few > 0 ? 1 : (a->B < a->N ? a->B : a->N);
  row_tiles = row_tiles < least ? least : row_tiles;
  const int64_t pairs = row_tiles * a->heads;
  int64_t splits = pairs > 0 ? 256 / pairs : 1;
  const int64_t most = tiles / a->least;
  splits = splits > most ? most : splits;
  splits = splits < 1 ? 1 : splits;
  // Prompts that fill the card just once: the last rows see twice the tokens of the mean, so that
  // their tiles are cut in two where that is worth the join (one of 8192 tokens and 8 heads of one
  // query head: 215 -> 187 us; cutting chunks, whose tiles see about alike, costs 3%).
  if (!paged && splits == 1 && pairs <= 256 && tiles >= 64) {
    splits = 2;
    a->least = 32;
  }
  a->splits = (int)splits;
  if (splits == 1) return 0;
  return (size_t)splits * a->N * a->heads * a->group * (dim + 2) * sizeof(float);
}

__int128 tile_attention_threads(const TileAttentionArgs& a, int dim) {
  // the join's workgroups have 256 threads for 256 / (dim / 4) rows
  const int64_t join = a.splits > 1 ? (int64_t)tile_rows(dim) * (dim / 4) : 0;
  const int64_t main = (int64_t)a.splits * 64 * tile_waves(dim);
  return __int128(tile_numbers(a, dim)) * a.heads * (main > join ? main : join);
}

void tile_attention_place(TileAttentionArgs* a, int dim, void* workspace) {
  const size_t rows = (size_t)a->N * a->heads * a->group;
  a->part_o = (float*)workspace;
  a->part_ml = (float2*)(a->part_o + (size_t)a->splits * rows * dim);
}

namespace {

template <typename T, int D, bool kPaged>
hipError_t launch_dim(const TileAttentionArgs& a, hipStream_t st) {
  const int64_t groups = tile_numbers(a, D) * a.heads;
  hipLaunchKernelGGL((tile_attention_kernel<T, D, kPaged>), dim3((unsigned)(groups * a.splits)),
                     dim3(64 * tile_waves(D)), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  constexpr int kParts = tile_rows(D) / (256 / (D / 4));
  hipLaunchKernelGGL((tile_join_kernel<T, D, kPaged>), dim3((unsigned)(groups * kParts)), dim3(256),
                     0, st, a);
  return hipGetLastError();
}

template <typename T, bool kPaged>
hipError_t launch_type(const TileAttentionArgs& a, int dim, hipStream_t st) {
  if (dim == 64) return launch_dim<T, 64, kPaged>(a, st);
  if (dim == 128) return launch_dim<T, 128, kPaged>(a, st);
  return launch_dim<T, 256, kPaged>(a, st);
}

template <bool kPaged>
hipError_t launch(const TileAttentionArgs& a, int dim, KvType type, hipStream_t st) {
  if (a.N <= 0) return hipSuccess;
  return type == kFp16 ? launch_type<Fp16, kPaged>(a, dim, st)
                       : launch_type<Bf16, kPaged>(a, dim, st);
}

}  // namespace

hipError_t launch_prompt_attention(const TileAttentionArgs& a, int dim, KvType type,
                                   hipStream_t st) {
  return launch<false>(a, dim, type, st);
}

hipError_t launch_chunk_attention(const TileAttentionArgs& a, int dim, KvType type,
                                  hipStream_t st) {
  return launch<true>(a, dim, type, st);
}

}  // namespace sfx

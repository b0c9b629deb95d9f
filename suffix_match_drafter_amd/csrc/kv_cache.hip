// kv_cache.hip -- quantising K and V into the paged cache as they are written, and reading
// them back.
//
// Block scale.  For 32 tokens of one head with largest finite magnitude m the scale is the least
// 2^e with m <= 448 * 2^e (448 = 1.75 * 2^8 is e4m3's largest value), e within
// [kKvMinExp, kKvMaxExp].  A power of two costs nothing here: e4m3 is itself a floating-point
// type, so a finer scale would not add a bit, and x * 2^-e is exact in fp32, so a stored value
// has been rounded once, to nearest even (relative error at most 2^-4).
//
// Appending.  A write that starts inside a block finds live tokens before it.  The block's
// exponent becomes the larger of the old one and the one that the new tokens need; when it
// grows by d the live codes are multiplied by 2^-d and rounded again, which changes only those
// that become subnormal.  A write that starts on a block's first token sets the exponent
// afresh.  Tokens of the block after the written ones keep their bytes.
#include "kv_cache.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

namespace sfx {

namespace {

// 16-byte vectors that need only their elements' alignment (gfx950 loads and stores them at any
// address): inputs may be slices of a fused projection with odd strides.
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef unsigned u32_a2 __attribute__((aligned(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Elements travel in words: a pair of 16-bit ones or one of 32 bits.
//   codes: two words' (16-bit) or four words' (32-bit) values over a power of two as four codes,
//   without saturation; widen: the reverse, half `hi` of a word of codes; floats: as fp32.
struct Bf16 {
  static constexpr int kBytes = 2;
  static constexpr unsigned kInf = 0x7f80;
  static __device__ float value(unsigned bits) { return __uint_as_float(bits << 16); }
  static __device__ unsigned codes(const unsigned* w, float scale) {
    i16x2 r{0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[0]), scale,
                                                  false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[1]), scale,
                                                  true);
    return __builtin_bit_cast(unsigned, r);
  }
  static __device__ f32x2 floats(unsigned w) {
    return f32x2{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
  }
  template <bool kHi> static __device__ unsigned widen(unsigned codes, float scale) {
    return __builtin_bit_cast(unsigned,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, kHi));
  }
};
struct Fp16 {
  static constexpr int kBytes = 2;
  static constexpr unsigned kInf = 0x7c00;
  static __device__ float value(unsigned bits) {
    return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
  }
  static __device__ unsigned codes(const unsigned* w, float scale) {
    i16x2 r{0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2, w[0]), scale,
                                                 false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2, w[1]), scale, true);
    return __builtin_bit_cast(unsigned, r);
  }
  static __device__ f32x2 floats(unsigned w) {
    const f16x2 h = __builtin_bit_cast(f16x2, w);
    return f32x2{(float)h[0], (float)h[1]};
  }
  // by way of fp32: a value may be outside fp16's normal range
  template <bool kHi> static __device__ unsigned widen(unsigned codes, float scale) {
    const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8(codes, kHi);
    return __builtin_bit_cast(unsigned, f16x2{(_Float16)(x[0] * scale), (_Float16)(x[1] * scale)});
  }
};
struct Fp32 {
  static constexpr int kBytes = 4;
  static constexpr unsigned kInf = 0x7f800000;
  static __device__ float value(unsigned bits) { return __uint_as_float(bits); }
  static __device__ unsigned codes(const unsigned* w, float scale) {
    i16x2 r{0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[0]), __uint_as_float(w[1]),
                                                 scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[2]), __uint_as_float(w[3]),
                                                 scale, true);
    return __builtin_bit_cast(unsigned, r);
  }
};

template <typename T>
constexpr int kWords = T::kBytes * 4;  // of 16 elements

// Saturates to e4m3's range; a NaN stays one.
__device__ __forceinline__ float saturate(float y) {
  y = y > 448.f ? 448.f : y;
  return y < -448.f ? -448.f : y;
}

// Four codes of four values that may not fit.
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
  unsigned w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(a), saturate(b), 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(saturate(c), saturate(d), w, true);
}
template <typename T>
__device__ __forceinline__ unsigned codes_saturated(const unsigned* w, float inv) {
  if constexpr (T::kBytes == 2) {
    const f32x2 a = T::floats(w[0]), b = T::floats(w[1]);
    return codes4(a[0] * inv, a[1] * inv, b[0] * inv, b[1] * inv);
  } else {
    return codes4(__uint_as_float(w[0]) * inv, __uint_as_float(w[1]) * inv,
                  __uint_as_float(w[2]) * inv, __uint_as_float(w[3]) * inv);
  }
}

// Largest magnitude, as bits, of m and the element(s) of w: with the sign cleared a float's bits
// order as its value does, infinity and NaN last.
template <typename T>
__device__ __forceinline__ unsigned max_bits(unsigned m, unsigned w) {
  if constexpr (T::kBytes == 2) {
    const u16x2 a = __builtin_bit_cast(u16x2, m);
    const u16x2 b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(a, b));
  } else {
    w &= 0x7fffffffu;
    return m > w ? m : w;
  }
}
// The same leaving infinities and NaN out.
template <typename T>
__device__ __forceinline__ unsigned max_bits_finite(unsigned m, unsigned w) {
  if constexpr (T::kBytes == 2) {
    unsigned lo = w & 0x7fff, hi = w >> 16 & 0x7fff;
    lo = lo >= T::kInf ? 0 : lo;
    hi = hi >= T::kInf ? 0 : hi;
    return max_bits<T>(m, lo | hi << 16);
  } else {
    w &= 0x7fffffffu;
    return max_bits<T>(m, w >= T::kInf ? 0 : w);
  }
}
template <typename T>
__device__ __forceinline__ unsigned wave_max_bits(unsigned m) {
  if constexpr (T::kBytes == 2) {
    const unsigned hi = m >> 16;
    m &= 0xffff;
    m = m > hi ? m : hi;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const unsigned x = __shfl_xor(m, o);
    m = m > x ? m : x;
  }
  return __builtin_amdgcn_readfirstlane(m);
}

// Least e in range with m <= 448 * 2^e.  m = f * 2^x with f in [1, 2): 448 = 1.75 * 2^8.
__device__ __forceinline__ int needed_exp(float m) {
  const int bits = __float_as_int(m);
  int e = ((bits >> 23) & 255) - 127 - 8;
  if ((bits & 0x7fffff) > 0x600000) ++e;
  return e < kKvMinExp ? kKvMinExp : (e > kKvMaxExp ? kKvMaxExp : e);
}

// The element map of one 32-token block for lane (r, g): 16-byte chunk c of the block, element e.
// Keys: chunk c = (16-token half tt, slab j), all of token 16 tt + r, dims 64 j + 16 g + e.
// Values: chunk c = slab, tokens 16 j + 4 g + i and dims 32 c + 2 r + f of e = (f, j, i).
template <int D, bool kVal>
struct Map {
  static constexpr int kChunks = D / 32;
  static __device__ int token(int c, int e, int r, int g) {
    return kVal ? 16 * ((e >> 2) & 1) + 4 * g + (e & 3) : 16 * (c / (D / 64)) + r;
  }
  // byte offset of chunk c from the (page, head) base; tok0 = first token of the block in the page
  static __device__ int64_t offset(const KvCache& k, int c, int r, int g, int tok0) {
    if (kVal) return (int64_t)tok0 * D + c * 1024 + r * 64 + g * 16;
    return (int64_t)(c % (D / 64)) * k.page_size * 64 +
           (int64_t)(tok0 + 16 * (c / (D / 64)) + r) * 64 + g * 16;
  }
};

// A chunk's 16 elements in the codes' order from the words as loaded, and back.  Keys lie in that
// order already; for values `raw` holds token e's (= (j, i)) dim pair: in 16 bits one word each,
// in 32 bits words e and 8 + e.
template <typename T, bool kVal>
__device__ __forceinline__ void to_order(const unsigned (&raw)[kWords<T>],
                                         unsigned (&w)[kWords<T>]) {
  if constexpr (kVal && T::kBytes == 2) {
#pragma unroll
    for (int p = 0; p < 8; ++p)
      w[p] = __builtin_amdgcn_perm(raw[2 * (p & 3) + 1], raw[2 * (p & 3)],
                                   p < 4 ? 0x05040100u : 0x07060302u);
  } else {
#pragma unroll
    for (int p = 0; p < kWords<T>; ++p) w[p] = raw[p];
  }
}

// One wavefront per (request, 32-token block, tensor, head).  The block's values stay in
// registers between the maximum and the rounding, so the input is read once and the kernel is
// bounded by that traffic (prompts: 1.5 vector instructions an element in 16 bits) or by one
// dependent chain of loads (a few tokens: counts, page id, then inputs, old codes and scale
// together).  Measured: 8 prompts of 8192 tokens of 8 heads of 128 in bf16 78 us, 4.8 TB/s; 256
// drafts of 17 tokens 16 us, a single token for 4 requests 4 us.
template <typename T, int D, bool kVal>
__device__ void write_block(const KvMoveArgs& a, int b, int h, int block, int start, int count,
                            int lane) {
  constexpr int kChunks = Map<D, kVal>::kChunks, kB = T::kBytes, kW = kWords<T>;
  const KvCache& kc = a.c;
  const int per_page = kc.page_size / kKvBlock;
  const int pi = kv_page_of(kc, block);
  if (pi >= a.max_pages) return;
  const int page = a.page_table[(int64_t)b * a.max_pages + pi];
  if (page < 0 || page >= kc.num_pages) return;
  const int sub = block - pi * per_page, tok0 = sub * kKvBlock;
  const int64_t ph = (int64_t)page * kc.heads + h;
  uint8_t* codes = (kVal ? kc.v : kc.k) + ph * kc.page_size * D;
  float* scale = (kVal ? kc.v_scale : kc.k_scale) + ph * per_page + sub;
  const KvStrides& s = kVal ? a.vs : a.ks;
  const char* in = (const char*)(kVal ? a.v : a.k) + (b * s.batch + h * s.head) * kB;
  const int r = lane >> 2, g = lane & 3;
  const int rel = block * kKvBlock - start;  // input index of the block's first token
  const bool full = rel >= 0 && rel + kKvBlock <= count, live_before = rel < 0;
  auto is_new = [&](int tok) { return rel + tok >= 0 && rel + tok < count; };
  auto source = [&](int tok) {  // a row that can be read: one that is not new is cleared below
    const int j = rel + tok;
    return in + (int64_t)(j < 0 ? 0 : (j < count ? j : count - 1)) * s.token * kB;
  };

  // Old bytes: a 16-byte chunk of values mixes eight tokens and is read before it is written; one of
  // keys is a single token's and is read only when it moves to another scale.
  u32x4 old[kChunks];
  float old_scale = 0.f;
  if (kVal && !full)
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      old[c] = *(const u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0));
  if (live_before) old_scale = *scale;
  // the lane's eight tokens of values, the same in every chunk: their rows, which of them are new
  const char* row[8];
  unsigned fresh[8];
  if constexpr (kVal)
#pragma unroll
    for (int ji = 0; ji < 8; ++ji) {
      const int tok = Map<D, true>::token(0, ji, r, g);
      row[ji] = source(tok) + 2 * r * kB;
      fresh[ji] = full || is_new(tok) ? ~0u : 0;
    }
  unsigned w[kChunks][kW];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    unsigned raw[kW];
    if constexpr (kVal) {
#pragma unroll
      for (int ji = 0; ji < 8; ++ji) {
        if constexpr (kB == 2) {
          raw[ji] = *(const u32_a2*)(row[ji] + 32 * c * kB);
        } else {
          const u32x2 x = *(const u32x2_a4*)(row[ji] + 32 * c * kB);
          raw[ji] = x[0];
          raw[8 + ji] = x[1];
        }
      }
      if (!full)
#pragma unroll
        for (int e = 0; e < kW; ++e) raw[e] &= fresh[e & 7];
    } else {
      const int tok = Map<D, false>::token(c, 0, r, g);
      const char* p = source(tok) + (64 * (c % (D / 64)) + 16 * g) * kB;
#pragma unroll
      for (int i = 0; i < kW / 4; ++i) {
        u32x4 x;
        if constexpr (kB == 2)
          x = *(const u32x4_a2*)(p + 16 * i);
        else
          x = *(const u32x4_a4*)(p + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) raw[4 * i + e] = full || is_new(tok) ? x[e] : 0;
      }
    }
    to_order<T, kVal>(raw, w[c]);
  }
  unsigned mb = 0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int e = 0; e < kW; ++e) mb = max_bits<T>(mb, w[c][e]);
  mb = wave_max_bits<T>(mb);
  const bool special = mb >= T::kInf;  // an infinity or a NaN: the maximum is over the others
  if (special) {
    mb = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int e = 0; e < kW; ++e) mb = max_bits_finite<T>(mb, w[c][e]);
    mb = wave_max_bits<T>(mb);
  }
  const float m = T::value(mb);
  int e_new = needed_exp(m), e_old = e_new;
  if (live_before) {
    e_old = kv_exp_of(old_scale);
    e_new = e_old > e_new ? e_old : e_new;
  }
  const float sc = kv_pow2(e_new), inv = kv_pow2(-e_new), move = kv_pow2(e_old - e_new);
  const bool moved = e_old != e_new;
  const bool fits = !special && m <= 448.f * sc;
  if (!kVal && moved)
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      old[c] = *(const u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0));
  // Bytes to take from the new codes and, when the scale moved, from the old ones' new codes: of
  // values' words 4 f + j by j (tokens 16 j + 4 g + i); of keys all or none.
  unsigned take[2], carry[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    take[j] = carry[j] = 0;
    if constexpr (kVal)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        take[j] |= fresh[4 * j + i] & 0xffu << (8 * i);
        if (moved && rel + Map<D, true>::token(0, 4 * j + i, r, g) < 0) carry[j] |= 0xffu << (8 * i);
      }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    u32x4* at = (u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0));
    u32x4 q;
    if (fits) {
#pragma unroll
      for (int d = 0; d < 4; ++d) q[d] = T::codes(&w[c][d * kW / 4], sc);
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) q[d] = codes_saturated<T>(&w[c][d * kW / 4], inv);
    }
    if (full) {
      *at = q;
      continue;
    }
    if constexpr (!kVal) {
      const int tok = Map<D, false>::token(c, 0, r, g);
      take[0] = take[1] = is_new(tok) ? ~0u : 0;
      carry[0] = carry[1] = moved && rel + tok < 0 ? ~0u : 0;
    }
    if (moved) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(old[c][d], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(old[c][d], true);
        const unsigned y = codes4(lo[0] * move, lo[1] * move, hi[0] * move, hi[1] * move);
        old[c][d] = (old[c][d] & ~carry[d & 1]) | (y & carry[d & 1]);
      }
    }
    if (kVal || moved)
#pragma unroll
      for (int d = 0; d < 4; ++d) q[d] = (q[d] & take[d & 1]) | (old[c][d] & ~take[d & 1]);
    if (take[0] | take[1] | carry[0] | carry[1]) *at = q;
  }
  if (lane == 0 && (!live_before || moved)) *scale = sc;
}

// Unit of the grid for one wavefront: head fastest (a token's heads are adjacent in the input),
// then tensor, block and request.
struct Unit {
  int b, h, block;
  bool val;
};
__device__ __forceinline__ Unit unit_of(int heads, int nb) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // a scalar to the compiler
  unsigned u = blockIdx.x * kKvMoveWaves + wave;  // below 2^26 + 4
  Unit r;
  r.h = u % heads;
  u /= heads;
  r.val = u & 1;
  u >>= 1;
  r.block = u % nb;
  r.b = u / nb;
  return r;
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kKvMoveWaves) void kv_write_kernel(KvMoveArgs a, int nb) {
  const int lane = threadIdx.x & 63;
  const Unit u = unit_of(a.c.heads, nb);
  if (u.b >= a.B) return;
  const int start = a.start[u.b];
  int count = a.count ? a.count[u.b] : a.T;
  count = count > a.T ? a.T : count;
  if (start < 0 || count <= 0) return;
  const int64_t blk = (int64_t)start / kKvBlock + u.block;
  if (blk * kKvBlock >= (int64_t)start + count || blk >= (1 << 26)) return;
  if (u.val)
    write_block<T, D, true>(a, u.b, u.h, (int)blk, start, count, lane);
  else
    write_block<T, D, false>(a, u.b, u.h, (int)blk, start, count, lane);
}

// LDS of one wavefront of the read: 32 rows of up to 256 bytes, 16 apart so that the lanes' words of
// four rows fall on different banks.
template <typename T, int D>
struct ReadLds {
  static constexpr int kDims = D * T::kBytes < 256 ? D : 256 / T::kBytes;
  static constexpr int kRow = kDims * T::kBytes + 16;
  static constexpr int kVecs = kKvBlock * kRow / 16;
};

// The reverse: one wavefront per (request, 32-token block, tensor, head), zeros for rows past the
// count or on an unmapped page.  Bounded by the traffic, which is mostly the result's: 8 x 16384
// tokens of 8 heads of 128 in bf16 150 to 167 us, 4.5 to 5.0 TB/s (stored straight from the
// lanes that hold them, 4 bytes at a time, the values took it to 184 to 203).
template <typename T, int D, bool kVal>
__device__ void read_block(const KvMoveArgs& a, int b, int h, int64_t block, int start, int count,
                           int lane, u32x4* turn) {
  constexpr int kChunks = Map<D, kVal>::kChunks, kB = T::kBytes;
  const KvCache& kc = a.c;
  const int per_page = kc.page_size / kKvBlock;
  const int64_t rel = block * kKvBlock - start;
  const int r = lane >> 2, g = lane & 3;
  const KvStrides& s = kVal ? a.vs : a.ks;
  char* out = (char*)(kVal ? a.v : a.k) + (b * s.batch + h * s.head) * kB;
  u32x4 w[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) w[c] = u32x4{0, 0, 0, 0};
  float scale = 1.f;
  const int pi = block < (1 << 26) ? kv_page_of(kc, (int)block) : a.max_pages;
  if (rel < count && pi < a.max_pages) {
    const int page = a.page_table[(int64_t)b * a.max_pages + pi];
    if (page >= 0 && page < kc.num_pages) {
      const int sub = (int)block - pi * per_page;
      const int64_t ph = (int64_t)page * kc.heads + h;
      const int tok0 = sub * kKvBlock;
      const uint8_t* codes = (kVal ? kc.v : kc.k) + ph * kc.page_size * D;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        w[c] = *(const u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0));
      scale = kv_pow2(kv_exp_of((kVal ? kc.v_scale : kc.k_scale)[ph * per_page + sub]));
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    if constexpr (kVal) {
      // A lane has two dims of eight tokens: the block turns in LDS, a piece of whole rows at a
      // time, and goes out 16 bytes a lane.
      constexpr int kPiece = ReadLds<T, D>::kDims, kRow = ReadLds<T, D>::kRow;
      char* lds = (char*)turn;
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // tokens e = 2 q, 2 q + 1
        u32x2 even, odd;             // their words
        const unsigned lo = w[c][q >> 1], hi = w[c][2 + (q >> 1)];  // f = 0, 1
        if constexpr (kB == 2) {
          const unsigned x = q & 1 ? T::template widen<true>(lo, scale)
                                   : T::template widen<false>(lo, scale);
          const unsigned y = q & 1 ? T::template widen<true>(hi, scale)
                                   : T::template widen<false>(hi, scale);
          even[0] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          odd[0] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        } else {
          const f32x2 x = q & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(lo, true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8(lo, false);
          const f32x2 y = q & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(hi, true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8(hi, false);
          even = u32x2{__float_as_uint(x[0] * scale), __float_as_uint(y[0] * scale)};
          odd = u32x2{__float_as_uint(x[1] * scale), __float_as_uint(y[1] * scale)};
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int tok = Map<D, true>::token(c, 2 * q + k, r, g);
          char* p = lds + tok * kRow + (32 * c % kPiece + 2 * r) * kB;
          if constexpr (kB == 2)
            *(unsigned*)p = k ? odd[0] : even[0];
          else
            *(u32x2*)p = k ? odd : even;
        }
      }
      if ((c + 1) * 32 % kPiece == 0) {
        // one wavefront's own LDS: its accesses stay in order, the compiler must keep them so
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int kLanes = kPiece * kB / 16;  // of a row
#pragma unroll
        for (int t = 0; t < kKvBlock; t += 64 / kLanes) {
          const int tok = t + lane / kLanes, at = lane % kLanes * 16;
          const int64_t j = rel + tok;
          u32x4 v = *(const u32x4*)(lds + tok * kRow + at);
          v = j < count ? v : u32x4{0, 0, 0, 0};
          char* p = out + (j * s.token + 32 * (c + 1) - kPiece) * kB + at;
          if (j >= 0 && j < a.T) {
            if constexpr (kB == 2)
              *(u32x4_a2*)p = v;
            else
              *(u32x4_a4*)p = v;
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    } else {
      const int64_t j = rel + Map<D, false>::token(c, 0, r, g);
      char* p = out + (j * s.token + 64 * (c % (D / 64)) + 16 * g) * kB;
      if (j < 0 || j >= a.T) continue;
      const bool live = j < count;
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        u32x4 v;
        if constexpr (kB == 2) {
          v = u32x4{T::template widen<false>(w[c][2 * i], scale),
                    T::template widen<true>(w[c][2 * i], scale),
                    T::template widen<false>(w[c][2 * i + 1], scale),
                    T::template widen<true>(w[c][2 * i + 1], scale)};
        } else {
          const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8(w[c][i], false);
          const f32x2 y = __builtin_amdgcn_cvt_pk_f32_fp8(w[c][i], true);
          v = u32x4{__float_as_uint(x[0] * scale), __float_as_uint(x[1] * scale),
                    __float_as_uint(y[0] * scale), __float_as_uint(y[1] * scale)};
        }
        v = live ? v : u32x4{0, 0, 0, 0};
        if constexpr (kB == 2)
          *(u32x4_a2*)(p + 16 * i) = v;
        else
          *(u32x4_a4*)(p + 16 * i) = v;
      }
    }
  }
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kKvMoveWaves) void kv_read_kernel(KvMoveArgs a, int nb) {
  const int lane = threadIdx.x & 63;
  __shared__ u32x4 turn[kKvMoveWaves][ReadLds<T, D>::kVecs];
  const Unit u = unit_of(a.c.heads, nb);
  if (u.b >= a.B) return;
  u32x4* mine = turn[threadIdx.x >> 6];
  int start = a.start[u.b];
  int count = a.count ? a.count[u.b] : a.T;
  count = count > a.T ? a.T : count;
  if (start < 0) start = count = 0;  // no such token: zeros
  const int64_t block = (int64_t)start / kKvBlock + u.block;
  if (block * kKvBlock >= (int64_t)start + a.T) return;
  if (u.val)
    read_block<T, D, true>(a, u.b, u.h, block, start, count, lane, mine);
  else
    read_block<T, D, false>(a, u.b, u.h, block, start, count, lane, mine);
}

template <template <typename, int> class K>
hipError_t dispatch(const KvMoveArgs& a, int dim, KvType type, hipStream_t st) {
  if (a.B <= 0 || a.T <= 0) return hipSuccess;
  const int nb = (int)kv_blocks_of(a.T);
  const dim3 grid((unsigned)(kv_move_threads(a.B, a.T, a.c.heads) / (64 * kKvMoveWaves)));
  auto pick = [&](auto t) {
    using T = decltype(t);
    auto f = dim == 64 ? K<T, 64>::get() : dim == 128 ? K<T, 128>::get() : K<T, 256>::get();
    hipLaunchKernelGGL(f, grid, dim3(64 * kKvMoveWaves), 0, st, a, nb);
  };
  if (type == kBf16)
    pick(Bf16{});
  else if (type == kFp16)
    pick(Fp16{});
  else
    pick(Fp32{});
  return hipGetLastError();
}

template <typename T, int D> struct Write {
  static auto get() { return kv_write_kernel<T, D>; }
};
template <typename T, int D> struct Read {
  static auto get() { return kv_read_kernel<T, D>; }
};

}  // namespace

hipError_t launch_kv_write(const KvMoveArgs& a, int dim, KvType type, hipStream_t st) {
  return dispatch<Write>(a, dim, type, st);
}

hipError_t launch_kv_read(const KvMoveArgs& a, int dim, KvType type, hipStream_t st) {
  return dispatch<Read>(a, dim, type, st);
}

}  // namespace sfx

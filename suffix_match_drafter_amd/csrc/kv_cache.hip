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

constexpr int kWavesPerGroup = 4;

// 16-byte vectors that need only their elements' alignment (gfx950 loads and stores them at any
// address): inputs may be slices of a fused projection with odd strides.
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef unsigned u32_a2 __attribute__((aligned(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));

struct Bf16 {};
struct Fp16 {};
struct Fp32 {};

__device__ __forceinline__ float half_bits_to_float(unsigned short b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return (float)h;
}
__device__ __forceinline__ unsigned short float_to_half_bits(float x) {
  const _Float16 h = (_Float16)x;
  unsigned short b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}
__device__ __forceinline__ unsigned short float_to_bf16_bits(float x) {
  const __bf16 h = (__bf16)x;
  unsigned short b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}

template <typename T> struct Elem;
template <> struct Elem<Bf16> {
  static constexpr int kBytes = 2;
  static __device__ float lo(unsigned w) { return __uint_as_float(w << 16); }
  static __device__ float hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ unsigned pack(float a, float b) {
    return float_to_bf16_bits(a) | ((unsigned)float_to_bf16_bits(b) << 16);
  }
};
template <> struct Elem<Fp16> {
  static constexpr int kBytes = 2;
  static __device__ float lo(unsigned w) { return half_bits_to_float((unsigned short)w); }
  static __device__ float hi(unsigned w) { return half_bits_to_float((unsigned short)(w >> 16)); }
  static __device__ unsigned pack(float a, float b) {
    return float_to_half_bits(a) | ((unsigned)float_to_half_bits(b) << 16);
  }
};
template <> struct Elem<Fp32> {
  static constexpr int kBytes = 4;
};

// 16 consecutive elements as floats.
template <typename T>
__device__ __forceinline__ void load16(const char* p, float (&x)[16]) {
  if constexpr (Elem<T>::kBytes == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 w = *(const u32x4_a2*)(p + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = Elem<T>::lo(w[e]);
        x[8 * i + 2 * e + 1] = Elem<T>::hi(w[e]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 w = *(const u32x4_a4*)(p + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = __uint_as_float(w[e]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store16(char* p, const float (&x)[16]) {
  if constexpr (Elem<T>::kBytes == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = Elem<T>::pack(x[8 * i + 2 * e], x[8 * i + 2 * e + 1]);
      *(u32x4_a2*)(p + 16 * i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[4 * i + e]);
      *(u32x4_a4*)(p + 16 * i) = w;
    }
  }
}

template <typename T>
__device__ __forceinline__ void load2(const char* p, float& a, float& b) {
  if constexpr (Elem<T>::kBytes == 2) {
    const unsigned w = *(const u32_a2*)p;
    a = Elem<T>::lo(w);
    b = Elem<T>::hi(w);
  } else {
    const u32x2 w = *(const u32x2_a4*)p;
    a = __uint_as_float(w[0]);
    b = __uint_as_float(w[1]);
  }
}

template <typename T>
__device__ __forceinline__ void store2(char* p, float a, float b) {
  if constexpr (Elem<T>::kBytes == 2) {
    *(u32_a2*)p = Elem<T>::pack(a, b);
  } else {
    u32x2 w;
    w[0] = __float_as_uint(a);
    w[1] = __float_as_uint(b);
    *(u32x2_a4*)p = w;
  }
}

// Saturates to e4m3's range; a NaN stays one.
__device__ __forceinline__ float saturate(float y) {
  y = y > 448.f ? 448.f : y;
  return y < -448.f ? -448.f : y;
}

// Four codes of four scaled values.
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
  unsigned w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(a), saturate(b), 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(saturate(c), saturate(d), w, true);
}

__device__ __forceinline__ void values4(unsigned w, float (&x)[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  x[0] = lo[0];
  x[1] = lo[1];
  x[2] = hi[0];
  x[3] = hi[1];
}

// Least e in range with m <= 448 * 2^e.  m = f * 2^x with f in [1, 2): 448 = 1.75 * 2^8.
__device__ __forceinline__ int needed_exp(float m) {
  const int bits = __float_as_int(m);
  int e = ((bits >> 23) & 255) - 127 - 8;
  if ((bits & 0x7fffff) > 0x600000) ++e;
  return e < kKvMinExp ? kKvMinExp : (e > kKvMaxExp ? kKvMaxExp : e);
}

__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  return m;
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

// One wavefront per (request, 32-token block, tensor, head).  The block's values stay in
// registers between the maximum and the rounding, so the input is read once: the kernel is
// bounded by that traffic (prompts), or by one dependent chain of loads (a few tokens).
template <typename T, int D, bool kVal>
__device__ void write_block(const KvMoveArgs& a, int b, int h, int block, int start, int count,
                            int lane) {
  constexpr int kChunks = Map<D, kVal>::kChunks, kB = Elem<T>::kBytes;
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
  auto is_new = [&](int tok) { return rel + tok >= 0 && rel + tok < count; };
  float x[kChunks][16];
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    if constexpr (kVal) {
#pragma unroll
      for (int ji = 0; ji < 8; ++ji) {
        const int tok = Map<D, true>::token(c, ji, r, g);
        x[c][ji] = x[c][8 + ji] = 0.f;
        if (is_new(tok))
          load2<T>(in + ((int64_t)(rel + tok) * s.token + 32 * c + 2 * r) * kB, x[c][ji],
                   x[c][8 + ji]);
      }
    } else {
      const int tok = Map<D, false>::token(c, 0, r, g);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[c][e] = 0.f;
      if (is_new(tok))
        load16<T>(in + ((int64_t)(rel + tok) * s.token + 64 * (c % (D / 64)) + 16 * g) * kB,
                  x[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float ax = fabsf(x[c][e]);
      m = ax < __builtin_inff() ? fmaxf(m, ax) : m;  // NaN and infinities take no part
    }
  m = wave_max(m);
  const bool live_before = rel < 0;
  int e_new = needed_exp(m), e_old = e_new;
  if (live_before) {
    e_old = kv_exp_of(*scale);
    e_new = e_old > e_new ? e_old : e_new;
  }
  const float inv = kv_pow2(-e_new), move = kv_pow2(e_old - e_new);
  const bool full = rel >= 0 && rel + kKvBlock <= count, moved = e_old != e_new;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    u32x4* at = (u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0));
    u32x4 w;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      w[d] = codes4(x[c][4 * d] * inv, x[c][4 * d + 1] * inv, x[c][4 * d + 2] * inv,
                    x[c][4 * d + 3] * inv);
    if (full) {
      *at = w;
      continue;
    }
    // part of the block: merge with the bytes that are there
    unsigned fresh = 0, live = 0;  // per element of the chunk
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int tok = Map<D, kVal>::token(c, e, r, g);
      if (is_new(tok)) fresh |= 1u << e;
      if (rel + tok < 0 && moved) live |= 1u << e;
    }
    if (!(fresh | live)) continue;
    const u32x4 old = *at;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      float y[4];
      values4(old[d], y);
      const unsigned q = codes4(y[0] * move, y[1] * move, y[2] * move, y[3] * move);
      unsigned fm = 0, lm = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (fresh >> (4 * d + i) & 1) fm |= 0xffu << (8 * i);
        if (live >> (4 * d + i) & 1) lm |= 0xffu << (8 * i);
      }
      w[d] = (w[d] & fm) | (q & lm) | (old[d] & ~(fm | lm));
    }
    *at = w;
  }
  if (lane == 0 && (!live_before || moved)) *scale = kv_pow2(e_new);
}

// Unit u of the grid: head fastest (a token's heads are adjacent in the input), then tensor,
// block and request.
template <typename T, int D>
__global__ __launch_bounds__(64 * kWavesPerGroup) void kv_write_kernel(KvMoveArgs a, int nb) {
  const int lane = threadIdx.x & 63;
  int64_t u = (int64_t)blockIdx.x * kWavesPerGroup + (threadIdx.x >> 6);
  const int h = (int)(u % a.c.heads);
  u /= a.c.heads;
  const bool val = u & 1;
  u >>= 1;
  const int b = (int)(u / nb);
  if (b >= a.B) return;
  const int start = a.start[b];
  int count = a.count ? a.count[b] : a.T;
  count = count > a.T ? a.T : count;
  if (start < 0 || count <= 0) return;
  const int64_t blk = (int64_t)start / kKvBlock + u % nb;
  if (blk * kKvBlock >= (int64_t)start + count || blk >= (1 << 26)) return;
  const int block = (int)blk;
  if (val)
    write_block<T, D, true>(a, b, h, block, start, count, lane);
  else
    write_block<T, D, false>(a, b, h, block, start, count, lane);
}

// The reverse: one wavefront per (request, 32-token block, tensor, head), zeros for rows past the
// count or on an unmapped page.
template <typename T, int D, bool kVal>
__device__ void read_block(const KvMoveArgs& a, int b, int h, int64_t block, int start, int count,
                           int lane) {
  constexpr int kChunks = Map<D, kVal>::kChunks, kB = Elem<T>::kBytes;
  const KvCache& kc = a.c;
  const int per_page = kc.page_size / kKvBlock;
  const int64_t rel = block * kKvBlock - start;
  const int r = lane >> 2, g = lane & 3;
  const KvStrides& s = kVal ? a.vs : a.ks;
  char* out = (char*)(kVal ? a.v : a.k) + (b * s.batch + h * s.head) * kB;
  bool mapped = false;
  const uint8_t* codes = nullptr;
  float scale = 0.f;
  int tok0 = 0;
  const int pi = block < (1 << 26) ? kv_page_of(kc, (int)block) : a.max_pages;
  if (rel < count && pi < a.max_pages) {
    const int page = a.page_table[(int64_t)b * a.max_pages + pi];
    if (page >= 0 && page < kc.num_pages) {
      mapped = true;
      const int sub = (int)block - pi * per_page;
      const int64_t ph = (int64_t)page * kc.heads + h;
      tok0 = sub * kKvBlock;
      codes = (kVal ? kc.v : kc.k) + ph * kc.page_size * D;
      scale = kv_pow2(kv_exp_of((kVal ? kc.v_scale : kc.k_scale)[ph * per_page + sub]));
    }
  }
  u32x4 w[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    w[c] = mapped ? *(const u32x4*)(codes + Map<D, kVal>::offset(kc, c, r, g, tok0))
                  : u32x4{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    float x[16];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      float y[4];
      values4(w[c][d], y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * d + i] = y[i] * scale;
    }
    if constexpr (kVal) {
#pragma unroll
      for (int ji = 0; ji < 8; ++ji) {
        const int64_t j = rel + Map<D, true>::token(c, ji, r, g);
        const bool in = j < count;
        if (j >= 0 && j < a.T)
          store2<T>(out + (j * s.token + 32 * c + 2 * r) * kB, in ? x[ji] : 0.f,
                    in ? x[8 + ji] : 0.f);
      }
    } else {
      const int64_t j = rel + Map<D, false>::token(c, 0, r, g);
      if (j >= count)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
      if (j >= 0 && j < a.T)
        store16<T>(out + (j * s.token + 64 * (c % (D / 64)) + 16 * g) * kB, x);
    }
  }
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kWavesPerGroup) void kv_read_kernel(KvMoveArgs a, int nb) {
  const int lane = threadIdx.x & 63;
  int64_t u = (int64_t)blockIdx.x * kWavesPerGroup + (threadIdx.x >> 6);
  const int h = (int)(u % a.c.heads);
  u /= a.c.heads;
  const bool val = u & 1;
  u >>= 1;
  const int b = (int)(u / nb);
  if (b >= a.B) return;
  int start = a.start ? a.start[b] : 0;
  int count = a.count ? a.count[b] : a.T;
  count = count > a.T ? a.T : count;
  if (start < 0) start = count = 0;  // no such token: zeros
  const int64_t block = (int64_t)start / kKvBlock + u % nb;
  if (block * kKvBlock >= (int64_t)start + a.T) return;
  if (val)
    read_block<T, D, true>(a, b, h, block, start, count, lane);
  else
    read_block<T, D, false>(a, b, h, block, start, count, lane);
}

// Blocks that T tokens can touch, whatever the start.
int blocks_of(int T) { return (int)(((int64_t)T + kKvBlock - 2) / kKvBlock + 1); }

template <template <typename, int> class K>
hipError_t dispatch(const KvMoveArgs& a, int dim, KvType type, hipStream_t st) {
  if (a.B <= 0 || a.T <= 0) return hipSuccess;
  const int nb = blocks_of(a.T);
  const int64_t units = (int64_t)a.B * nb * 2 * a.c.heads;
  const dim3 grid((unsigned)((units + kWavesPerGroup - 1) / kWavesPerGroup));
  auto pick = [&](auto t) {
    using T = decltype(t);
    auto f = dim == 64 ? K<T, 64>::get() : dim == 128 ? K<T, 128>::get() : K<T, 256>::get();
    hipLaunchKernelGGL(f, grid, dim3(64 * kWavesPerGroup), 0, st, a, nb);
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

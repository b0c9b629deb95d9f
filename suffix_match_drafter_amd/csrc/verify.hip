// verify.hip -- verification of drafted tokens against the target's logits from given random
// numbers.
//
// The drafter proposes tokens, not distributions, so slot i's draft d is a point mass and the
// rule that leaves the target's distribution unchanged is: accept d when u_i < p_i(d); at the
// first rejection draw from p_i with d removed and renormalised; when every drafted token is
// accepted draw one more from the next row.  With w_j = exp((l_j - max l) / T) and Z = sum w,
//   accept:  u Z < w_d
//   draw:    the least j with w_0 + ... + w_j > u Z',  w_d = 0 after a rejection, Z' its sum.
// T = 0 (or less, or NaN) is greedy: a draft is accepted when it is the row's largest logit (the
// lowest index of equals), which is also what is drawn.  A NaN logit counts as -inf.
//
// Precision.  The statistics of all rows come from one pass in fp32 (memory-bound).  Both
// comparisons decide a token, so neither is left to rounding: a test whose two sides are within
// the fp32 pass's error bound is redone in fp64, and the row that is drawn from is summed
// and searched in fp64.
#include "verify.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

namespace sfx {

namespace {

constexpr int kStatThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kPickWaves = kPickThreads / 64;
constexpr int kMaxRows = 33;  // k + 1

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ float from_half(unsigned short b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return (float)h;
}

// A logit as the sums take it: NaN is -inf; +inf becomes the largest float, so that equal
// infinities differ by 0 and share the row.
__device__ __forceinline__ float clean(float x) {
  return x == x ? fminf(x, 3.402823466e38f) : -__builtin_inff();
}

struct Bf16 {
  static constexpr int kBytes = 2;
  static __device__ float get(const void* p, int64_t i) {
    return clean(__uint_as_float((unsigned)((const unsigned short*)p)[i] << 16));
  }
  static __device__ void get8(const void* p, int64_t i, float (&x)[8]) {
    const u32x4 w = *(const u32x4_a2*)((const unsigned short*)p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = clean(__uint_as_float(w[e] << 16));
      x[2 * e + 1] = clean(__uint_as_float(w[e] & 0xffff0000u));
    }
  }
};
struct Fp16 {
  static constexpr int kBytes = 2;
  static __device__ float get(const void* p, int64_t i) {
    return clean(from_half(((const unsigned short*)p)[i]));
  }
  static __device__ void get8(const void* p, int64_t i, float (&x)[8]) {
    const u32x4 w = *(const u32x4_a2*)((const unsigned short*)p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = clean(from_half((unsigned short)w[e]));
      x[2 * e + 1] = clean(from_half((unsigned short)(w[e] >> 16)));
    }
  }
};
struct Fp32 {
  static constexpr int kBytes = 4;
  static __device__ float get(const void* p, int64_t i) { return clean(((const float*)p)[i]); }
  static __device__ void get8(const void* p, int64_t i, float (&x)[8]) {
    const u32x4 w = *(const u32x4_a4*)((const float*)p + i);
    const u32x4 v = *(const u32x4_a4*)((const float*)p + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = clean(__uint_as_float(w[e]));
      x[4 + e] = clean(__uint_as_float(v[e]));
    }
  }
};

__device__ __forceinline__ int clamp_valid(const VerifyArgs& a, int b) {
  const int nv = a.num_valid ? a.num_valid[b] : a.k;
  return nv < 0 ? 0 : (nv > a.k ? a.k : nv);
}
__device__ __forceinline__ float temperature(const VerifyArgs& a, int b) {
  return a.temperature ? a.temperature[b] : 1.f;
}
// log2(e) / T and 1 / T, finite and above 0 whatever T > 0 is, so that 0 and -inf times it stay
// 0 and -inf.
__device__ __forceinline__ float inv_log2(float t) {
  return fminf(fmaxf(1.4426950408889634f / t, 1e-30f), 1e30f);
}
__device__ __forceinline__ double inv64(float t) { return fmax(1.0 / (double)t, 1e-300); }

__device__ __forceinline__ float fmerge(float m, float s, float m2, float s2, float c, float mm) {
  const float z = mm == -__builtin_inff() ? 0.f : mm;
  return s * __builtin_amdgcn_exp2f((m - z) * c) + s2 * __builtin_amdgcn_exp2f((m2 - z) * c);
}

// One part of one row: largest logit, its lowest index, sum of exponentials.  Memory-bound.
template <typename T>
__global__ __launch_bounds__(kStatThreads) void verify_stats_kernel(VerifyArgs a) {
  const int part = (int)(blockIdx.x % a.parts);
  const int64_t rowid = blockIdx.x / a.parts;  // slot-major
  const int slot = (int)(rowid / a.B), b = (int)(rowid % a.B);
  if (slot > clamp_valid(a, b)) return;
  const char* row = (const char*)a.logits +
                    ((int64_t)b * a.batch_stride + slot * a.slot_stride) * T::kBytes;
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  const float c = greedy ? 1.f : inv_log2(temp);
  const int j0 = part * a.part_size;
  const int j1 = a.V - j0 < a.part_size ? a.V : j0 + a.part_size;
  float m = -__builtin_inff(), s = 0.f;
  int at = 0x7fffffff;
  for (int j = j0 + (int)threadIdx.x * 8; j < j1; j += kStatThreads * 8) {
    float x[8];
    if (j + 8 <= j1) {
      T::get8(row, j, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = j + e < j1 ? T::get(row, j + e) : -__builtin_inff();
    }
    float t = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) t = fmaxf(t, x[e]);
    if (t > m) {
      s *= __builtin_amdgcn_exp2f((m - t) * c);
      m = t;
#pragma unroll
      for (int e = 7; e >= 0; --e)
        if (x[e] == t) at = j + e;
    }
    if (!greedy) {
      const float z = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((x[e] - z) * c);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
    const int at2 = __shfl_xor(at, o);
    const float mm = fmaxf(m, m2);
    s = fmerge(m, s, m2, s2, c, mm);
    at = m2 > m || (m2 == m && at2 < at) ? at2 : at;
    m = mm;
  }
  __shared__ VerifyPart w[kStatThreads / 64];
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = VerifyPart{m, s, at, 0};
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kStatThreads / 64; ++i) {
      const float mm = fmaxf(m, w[i].m);
      s = fmerge(m, s, w[i].m, w[i].s, c, mm);
      at = w[i].m > m || (w[i].m == m && w[i].at < at) ? w[i].at : at;
      m = mm;
    }
    a.part[((int64_t)b * (a.k + 1) + slot) * a.parts + part] = VerifyPart{m, s, at, 0};
  }
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ double weight64(float x, float m, double inv) {
  return exp(((double)x - (double)m) * inv);
}

// Sum of the weights of [j0, j1), one wavefront, `skip` left out.
template <typename T>
__device__ double wave_range64(const char* row, int j0, int j1, float m, double inv, int skip,
                               int lane) {
  double s = 0.0;
  for (int j = j0 + lane * 8; j < j1; j += 512) {
    float x[8];
    if (j + 8 <= j1) {
      T::get8(row, j, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = j + e < j1 ? T::get(row, j + e) : -__builtin_inff();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s += j + e == skip ? 0.0 : weight64(x[e], m, inv);
  }
  return wave_sum64(s);
}

// Segment w of [j0, j1) in kPickWaves equal ones.
__device__ __forceinline__ int seg_at(int j0, int j1, int w) {
  const int len = (j1 - j0 + kPickWaves - 1) / kPickWaves;
  const int64_t j = (int64_t)j0 + (int64_t)len * w;
  return j < j1 ? (int)j : j1;
}

// One workgroup per request: the tests in order, then the draw from the row they end at.
template <typename T>
__global__ __launch_bounds__(kPickThreads) void verify_pick_kernel(VerifyArgs a) {
  __shared__ float row_m[kMaxRows];
  __shared__ int row_at[kMaxRows], verdict[kMaxRows];
  __shared__ double seg[kPickWaves];
  __shared__ int token;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nv = clamp_valid(a, b);
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  const float c = greedy ? 1.f : inv_log2(temp);
  const double inv = greedy ? 1.0 : inv64(temp);
  const char* rows = (const char*)a.logits + (int64_t)b * a.batch_stride * T::kBytes;
  auto row_of = [&](int i) { return rows + i * a.slot_stride * T::kBytes; };
  if (tid <= nv) {
    const VerifyPart* p = a.part + ((int64_t)b * (a.k + 1) + tid) * a.parts;
    float m = p[0].m;
    int at = p[0].at;
    for (int i = 1; i < a.parts; ++i)
      if (p[i].m > m) {
        m = p[i].m;
        at = p[i].at;
      }
    row_m[tid] = m;
    row_at[tid] = at;
    int v = 0;
    if (tid < nv && m > -__builtin_inff()) {
      const int d = a.draft[(int64_t)b * a.k + tid];
      if (d >= 0 && d < a.V) {
        if (greedy) {
          v = at == d;
        } else {
          float z = 0.f;
          for (int i = 0; i < a.parts; ++i)
            z += p[i].s * __builtin_amdgcn_exp2f((p[i].m - m) * c);
          const float w = __builtin_amdgcn_exp2f((T::get(row_of(tid), d) - m) * c);
          const float uz = a.u_accept[(int64_t)b * a.k + tid] * z;
          // the fp32 sides are off by less than 2^-16 of themselves where w is not tiny
          v = fabsf(uz - w) <= (uz + w) * 0x1p-14f + 0x1p-60f ? 2 : (uz < w ? 1 : 0);
        }
      }
    }
    verdict[tid] = v;
  }
  __syncthreads();
  int n = 0;
  for (; n < nv; ++n) {
    int v = verdict[n];
    if (v == 2) {
      const double s = wave_range64<T>(row_of(n), seg_at(0, a.V, wave), seg_at(0, a.V, wave + 1),
                                       row_m[n], inv, -1, lane);
      if (lane == 0) seg[wave] = s;
      __syncthreads();
      double z = 0.0;
      for (int w = 0; w < kPickWaves; ++w) z += seg[w];
      __syncthreads();
      const int d = a.draft[(int64_t)b * a.k + n];
      v = (double)a.u_accept[(int64_t)b * a.k + n] * z <
          weight64(T::get(row_of(n), d), row_m[n], inv);
    }
    if (!v) break;
  }
  int pick = -1;
  if (row_m[n] > -__builtin_inff()) {
    pick = row_at[n];
    if (!greedy) {
      const int d = n < nv ? a.draft[(int64_t)b * a.k + n] : -1;
      const char* row = row_of(n);
      const float m = row_m[n];
      int j0 = 0, j1 = a.V;
      double base = 0.0, t = 0.0;
      bool none = false;
      for (int level = 0; level < 2; ++level) {
        const double s = wave_range64<T>(row, seg_at(j0, j1, wave), seg_at(j0, j1, wave + 1), m,
                                         inv, d, lane);
        if (lane == 0) seg[wave] = s;
        __syncthreads();
        if (level == 0) {
          double z = 0.0;
          for (int w = 0; w < kPickWaves; ++w) z += seg[w];
          t = (double)a.u_sample[b] * z;
          none = !(z > 0.0);  // the rejected draft was all there was
        }
        // the segment whose sums pass t; the last that holds anything if rounding hides it
        int at = -1;
        double before = base, run = base;
        for (int w = 0; w < kPickWaves; ++w) {
          if (seg[w] > 0.0) {
            at = w;
            before = run;
            run += seg[w];
            if (run > t) break;
          }
        }
        __syncthreads();
        if (at < 0) at = 0;
        base = before;
        const int s0 = seg_at(j0, j1, at), s1 = seg_at(j0, j1, at + 1);
        j0 = s0;
        j1 = s1;
      }
      if (none) {
        pick = row_at[n];
      } else {
        if (wave == 0) {
          int found = -1;
          for (int j = j0; j < j1; j += 64) {
            double w = 0.0;
            if (j + lane < j1 && j + lane != d) w = weight64(T::get(row, j + lane), m, inv);
            double inc = w;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
              const double y = __shfl_up(inc, o);
              if (lane >= o) inc += y;
            }
            const unsigned long long some = __ballot(w > 0.0);
            const unsigned long long hit = __ballot(w > 0.0 && base + inc > t);
            if (some) found = j + 63 - __clzll(some);
            if (hit) {
              found = j + __ffsll((long long)hit) - 1;
              break;
            }
            base += __shfl(inc, 63);
          }
          if (lane == 0) token = found;
        }
        __syncthreads();
        pick = token;
      }
    }
  }
  if (tid <= a.k)
    a.sampled[(int64_t)b * (a.k + 1) + tid] =
        tid < n ? a.draft[(int64_t)b * a.k + tid] : (tid == n ? pick : -1);
  if (tid == 0) a.num_accepted[b] = n;
}

template <typename T>
hipError_t launch_type(const VerifyArgs& a, hipStream_t st) {
  const int64_t groups = (int64_t)a.B * (a.k + 1) * a.parts;
  hipLaunchKernelGGL(verify_stats_kernel<T>, dim3((unsigned)groups), dim3(kStatThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel<T>, dim3((unsigned)a.B), dim3(kPickThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t verify_plan(VerifyArgs* a) {
  // parts of at least 16K logits, enough of them to fill 256 CUs four times over
  const int64_t rows = (int64_t)a->B * (a->k + 1);
  int64_t parts = rows > 0 ? (1024 + rows - 1) / rows : 1;
  const int64_t most = ((int64_t)a->V + 16383) / 16384;
  parts = parts > most ? most : parts;
  parts = parts < 1 ? 1 : parts;
  const int64_t size = (a->V + parts - 1) / parts;
  a->part_size = (int32_t)((size + 7) / 8 * 8);
  a->parts = (int32_t)((a->V + a->part_size - 1) / a->part_size);
  if (a->parts < 1) a->parts = 1;
  return (size_t)rows * a->parts * sizeof(VerifyPart);
}

hipError_t launch_verify(const VerifyArgs& a, KvType type, hipStream_t st) {
  if (a.B <= 0) return hipSuccess;
  if (type == kBf16) return launch_type<Bf16>(a, st);
  if (type == kFp16) return launch_type<Fp16>(a, st);
  return launch_type<Fp32>(a, st);
}

}  // namespace sfx

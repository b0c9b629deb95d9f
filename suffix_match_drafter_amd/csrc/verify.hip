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
// Precision.  A row's statistics (maximum, sum) come from one pass in fp32, bounded by the
// reading of the logits.  Both comparisons decide a token, so neither is left to rounding: a
// test whose two sides are within the fp32 pass's error bound is redone in fp64, and the row that
// is drawn from is summed and searched in fp64.
//
// Work.  Rows past the first rejection decide nothing.  Large calls go through the slots in four
// launches (0, 1-2, 3-6, 7-k), each over the requests that are still undecided, so that few rows are
// read in vain and each launch fills the card.  Small calls, where four launches would cost more
// than the rows they save, read all rows in parts at once.
//
// Measured, k = 8 and V = 151936 in bf16: B = 1 20 us, B = 16 33, B = 64 63; B = 256, k = 16 153 us
// when 64% of the drafted tokens are accepted, of which 110 read 965 rows of 4352 (2.7 TB/s; 720
// rows would do) and 40 sum and search the drawn ones.
#include "verify.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

namespace sfx {

namespace {

constexpr int kPartThreads = 256;   // workgroup of a part of a row
constexpr int kRowThreads = 1024;   // workgroup of a whole row, and of a request's draw
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kMaxRows = 33;        // k + 1
// Vocabularies up to this go in one launch: 12-14 us a call at B = 4, k = 8 and V = 1024-4096 where
// two launches take 17, 25.6 against 37.1 at B = 256, k = 32, V = 4096; at V = 8192 17.4 against
// 16.9 and 34.3 against 45.9, at 16384 25 against 17.
constexpr int kSmallV = 4096;
constexpr int kPhaseThreads = 256;  // workgroup of a phase after the first
constexpr int kPhaseGroups = 1024;  // four on each of 256 CUs

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ float from_half(unsigned short b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return (float)h;
}

// A logit as the sums take it: NaN is -inf (a maximum drops it).
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -__builtin_inff()); }

// x - m for x <= m.  Equal infinities differ by 0: logits of +inf share their row, and what is
// finite beside them weighs nothing at any temperature.
__device__ __forceinline__ float below(float x, float m) { return x == m ? 0.f : x - m; }

// One logit, and eight as they lie in memory (any alignment of their type) and as floats.
struct Bf16 {
  static constexpr int kBytes = 2;
  struct Raw {
    u32x4 w;
  };
  static __device__ float get(const void* p, int64_t i) {
    return __uint_as_float((unsigned)((const unsigned short*)p)[i] << 16);
  }
  static __device__ Raw raw8(const void* p, int64_t i) {
    return Raw{*(const u32x4_a2*)((const unsigned short*)p + i)};
  }
  static __device__ void floats(const Raw& r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(r.w[e] << 16);
      x[2 * e + 1] = __uint_as_float(r.w[e] & 0xffff0000u);
    }
  }
};
struct Fp16 {
  static constexpr int kBytes = 2;
  struct Raw {
    u32x4 w;
  };
  static __device__ float get(const void* p, int64_t i) {
    return from_half(((const unsigned short*)p)[i]);
  }
  static __device__ Raw raw8(const void* p, int64_t i) {
    return Raw{*(const u32x4_a2*)((const unsigned short*)p + i)};
  }
  static __device__ void floats(const Raw& r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = from_half((unsigned short)r.w[e]);
      x[2 * e + 1] = from_half((unsigned short)(r.w[e] >> 16));
    }
  }
};
struct Fp32 {
  static constexpr int kBytes = 4;
  struct Raw {
    u32x4 w, v;
  };
  static __device__ float get(const void* p, int64_t i) { return ((const float*)p)[i]; }
  static __device__ Raw raw8(const void* p, int64_t i) {
    return Raw{*(const u32x4_a4*)((const float*)p + i),
               *(const u32x4_a4*)((const float*)p + i + 4)};
  }
  static __device__ void floats(const Raw& r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __uint_as_float(r.w[e]);
      x[4 + e] = __uint_as_float(r.v[e]);
    }
  }
};

template <typename T>
__device__ __forceinline__ float logit(const void* row, int64_t j) {
  return clean(T::get(row, j));
}

// Calls f(eight logits, index of the first) for j, j + step, ... below j1; missing ones are -inf.
// Loads run a batch ahead of the work on them, in two sets of registers that take turns (a copy
// from one to the other would wait for the loads).
template <typename T, int kBatch, typename F>
__device__ __forceinline__ void each8(const char* row, int j, int j1, int step, F&& f) {
  const int batch = kBatch * step, reach = (kBatch - 1) * step + 8;
  float x[8];
  if (j + reach <= j1) {
    typename T::Raw a[kBatch], b[kBatch];
    auto load = [&](typename T::Raw (&r)[kBatch], int at) {
      // past the end: any place inside, not used
      const int from = at + reach <= j1 ? at : j;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r[k] = T::raw8(row, from + k * step);
    };
    auto work = [&](const typename T::Raw (&r)[kBatch], int at) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        T::floats(r[k], x);
        f(x, at + k * step);
      }
    };
    load(a, j);
    for (;;) {
      load(b, j + batch);
      work(a, j);
      j += batch;
      if (j + reach > j1) break;
      load(a, j + batch);
      work(b, j);
      j += batch;
      if (j + reach > j1) break;
    }
  }
  for (; j < j1; j += step) {
    if (j + 8 <= j1) {
      T::floats(T::raw8(row, j), x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = j + e < j1 ? T::get(row, j + e) : -__builtin_inff();
    }
    f(x, j);
  }
}

__device__ __forceinline__ int clamp_valid(const VerifyArgs& a, int b) {
  const int nv = a.num_valid ? a.num_valid[b] : a.k;
  return nv < 0 ? 0 : (nv > a.k ? a.k : nv);
}
__device__ __forceinline__ float temperature(const VerifyArgs& a, int b) {
  return a.temperature ? a.temperature[b] : 1.f;
}
// log2(e) / T and 1 / T, finite and above 0 whatever T > 0 is, so that 0 and -inf times it stay
// 0 and -inf.  In fp32 the range is narrower than T's; beyond it the fp32 sums decide nothing
// (test_slot).
constexpr float kInvLo = 1e-30f, kInvHi = 1e30f;
__device__ __forceinline__ float inv_log2(float t) {
  return fminf(fmaxf(1.4426950408889634f / t, kInvLo), kInvHi);
}
__device__ __forceinline__ double inv64(float t) { return fmax(1.0 / (double)t, 1e-300); }

// Two parts of a row as one; of equal largest logits the lowest index.
__device__ __forceinline__ VerifyPart join(const VerifyPart& p, const VerifyPart& q, float c) {
  const float m = fmaxf(p.m, q.m);
  return VerifyPart{m, p.s * __builtin_amdgcn_exp2f(below(p.m, m) * c) +
                           q.s * __builtin_amdgcn_exp2f(below(q.m, m) * c),
                    q.m > p.m || (q.m == p.m && q.at < p.at) ? q.at : p.at, 0};
}

// Largest logit, its lowest index and the sum of exponentials of the logits that a wavefront's
// lanes take: eight each at j, j + step, ... below j1.  The result is every lane's.
template <typename T, int kBatch, bool kClean>
__device__ __forceinline__ VerifyPart wave_stats(const char* row, int j, int j1, int step,
                                                 bool greedy, float c) {
  float m = -__builtin_inff(), s = 0.f;
  int at = 0x7fffffff;
  each8<T, kBatch>(row, j, j1, step, [&](float (&x)[8], int j) {
    if (kClean)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = clean(x[e]);
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
      for (int e = 0; e < 8; ++e)
        x[e] = __builtin_amdgcn_exp2f((kClean ? below(x[e], z) : x[e] - z) * c);
      s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    }
  });
  VerifyPart r{m, s, at, 0};
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1)
    r = join(r, VerifyPart{__shfl_xor(r.m, o), __shfl_xor(r.s, o), __shfl_xor(r.at, o), 0}, c);
  return r;
}

// Taken as they come, a NaN or +inf among the logits makes the sum a NaN or the maximum infinite;
// then, and only then, they are cleaned and summed again.
__device__ __forceinline__ bool to_clean(const VerifyPart& r) {
  return !(r.s < __builtin_inff()) || r.m == __builtin_inff();
}

template <typename T, int N, bool kClean>
__device__ __forceinline__ VerifyPart group_stats(const char* row, int j0, int j1, bool greedy, float c,
                                  VerifyPart* w) {
  const VerifyPart mine = wave_stats<T, 4, kClean>(row, j0 + (int)threadIdx.x * 8, j1, N * 8,
                                                   greedy, c);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = mine;
  __syncthreads();
  VerifyPart r = w[0];
  for (int i = 1; i < N / 64; ++i) r = join(r, w[i], c);
  return r;
}

// Logits [j0, j1) of a row by a workgroup of N threads; the result is every thread's.
template <typename T, int N>
__device__ __forceinline__ VerifyPart row_stats(const char* row, int j0, int j1, bool greedy, float c) {
  __shared__ VerifyPart w[N / 64];
  VerifyPart r = group_stats<T, N, false>(row, j0, j1, greedy, c, w);
  if (to_clean(r)) r = group_stats<T, N, true>(row, j0, j1, greedy, c, w);
  return r;
}

__device__ __forceinline__ const char* row_ptr(const VerifyArgs& a, int b, int slot, int bytes) {
  return (const char*)a.logits + ((int64_t)b * a.batch_stride + slot * a.slot_stride) * bytes;
}

// ---------------------------------------------------------------- fp64 weights
// exp by a table of 2^(i/256) and a polynomial over 1/256 of an octave, |z| <= ln 2 / 512:
//   2^(n/256 + f/256) = 2^(n div 256) T[n mod 256] (1 + z + z^2/2 + z^3/6),  z = f ln 2 / 256,
// within 2^-42 of the function.  The search for the drawn token is bounded by these instructions
// (19 a logit, 40 us for 256 rows of 151936 with the launch; 27 a logit, with 32 entries, two more
// terms and a select, took 11 us more).  Logits more than 700 T below the largest weigh e^-700
// here, whatever they are: what they add is far below a draw's resolution unless the draw is below
// kTiny, which is done again with the exact function.
constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer
constexpr double kZ = 0.69314718055994530942 / 256;
constexpr int kTable = 256;
constexpr double kTiny = 0x1p-900;  // above 2^30 times e^-700

struct Weights64 {
  const double* table;  // kTable entries in LDS
  double k;             // 256 log2(e) / T
  double m;
  double lo;            // -700 T
};

__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < kTable) table[threadIdx.x] = exp2((double)threadIdx.x / kTable);
}

__device__ __forceinline__ Weights64 weights64(const double* table, float m, float temp,
                                               bool greedy) {
  const double inv = greedy ? 1.0 : inv64(temp);
  return Weights64{table, inv * (kTable * 1.4426950408889634074), (double)m, -700.0 / inv};
}

// Sum of four weights, stage by stage: each weight is one chain of dependent instructions.  The
// maximum takes -inf and NaN to the floor too, at any temperature (+inf does not get here).
__device__ __forceinline__ double weights4(const Weights64& w, const float* x) {
  double f[4], p[4], ts[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double d = fmax((double)x[e] - w.m, w.lo);
    const double t = fma(d, w.k, kMagic);
    const int n = (int)__double_as_longlong(t);  // low word: the integer
    f[e] = fma(d, w.k, -(t - kMagic));
    const double s = w.table[n & (kTable - 1)];
    ts[e] = __hiloint2double(__double2hiint(s) + ((n & ~(kTable - 1)) << 12),
                             __double2loint(s));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = fma(f[e], kZ * kZ * kZ / 6, kZ * kZ / 2);
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = fma(f[e], p[e], kZ);
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = fma(ts[e], p[e] * f[e], ts[e]);
  return (p[0] + p[1]) + (p[2] + p[3]);
}

// The same to the last weight above 0 that fp64 has: for draws at the very start of a row.
__device__ __forceinline__ double weight64_full(float x, float m, double inv) {
  return x == m ? 1.0 : exp(((double)x - (double)m) * inv);
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Sum of the weights of [j0, j1) (as of weights4; `skip` counts as masked), one wavefront.  Where
// the largest logit is +inf, its equals weigh 1 and are counted.
template <typename T>
__device__ __forceinline__ double wave_range64(const char* row, int j0, int j1, const Weights64& w, int skip,
                               int lane) {
  double s = 0.0;
  if (w.m == (double)__builtin_inff()) {
    for (int j = j0 + lane; j < j1; j += 64)
      if (j != skip && T::get(row, j) == __builtin_inff()) s += 1.0;
    return wave_sum64(s);
  }
  each8<T, 4 / T::kBytes>(row, j0 + lane * 8, j1, 512, [&](float (&x)[8], int j) {
    if ((unsigned)(skip - j) < 8u)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e == skip) x[e] = -__builtin_inff();
    s += weights4(w, x);
    s += weights4(w, x + 4);
  });
  return wave_sum64(s);
}

// Segment w of [j0, j1) in `of` equal ones.
__device__ __forceinline__ int seg_at(int j0, int j1, int w, int of) {
  const int len = (j1 - j0 + of - 1) / of;
  const int64_t j = (int64_t)j0 + (int64_t)len * w;
  return j < j1 ? (int)j : j1;
}

// ---------------------------------------------------------------- tests
enum { kReject = 0, kAccept = 1, kClose = 2 };

// The test of slot `slot` from its row's fp32 statistics; `groups`: groups of eight logits that
// one thread of the pass added up in turn.
//
// Errors, in units of 2^-23: an exponent x is rounded three times, 1.04 |x| of its weight, and
// the function's own 1; over a sum that averages to at most 1.04 log2 V (31).  Each group may add
// a rounding and, when the maximum moved, a rescaling (3).  The joins of threads and parts fit the
// rest of 64.  Weights below 2^-126 are lost: under 2^-60 of any sum.
template <typename T>
__device__ int test_slot(const VerifyArgs& a, int b, int slot, const VerifyPart& p, bool greedy,
                         float c, int groups) {
  if (!(p.m > -__builtin_inff())) return kReject;
  const int d = a.draft[(int64_t)b * a.k + slot];
  if (d < 0 || d >= a.V) return kReject;
  if (greedy) return p.at == d ? kAccept : kReject;
  if (c <= kInvLo || c >= kInvHi) return kClose;  // another temperature than the request's
  const float x = below(logit<T>(row_ptr(a, b, slot, T::kBytes), d), p.m) * c;
  const float w = __builtin_amdgcn_exp2f(x);
  const float uz = a.u_accept[(int64_t)b * a.k + slot] * p.s;
  const float off = uz * (3 * groups + 64) + w * (1.04f * fminf(-x, 200.f) + 4);
  if (fabsf(uz - w) <= off * 0x1p-23f + 0x1p-60f) return kClose;
  return uz < w ? kAccept : kReject;
}

// The same in fp64, by a whole workgroup of kRowThreads; seg: kRowWaves doubles of LDS.
template <typename T>
__device__ bool test_close(const VerifyArgs& a, int b, int slot, const Weights64& w, float m,
                           double inv, double* seg) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const char* row = row_ptr(a, b, slot, T::kBytes);
  const double s = wave_range64<T>(row, seg_at(0, a.V, wave, kRowWaves),
                                   seg_at(0, a.V, wave + 1, kRowWaves), w, -1, lane);
  __syncthreads();
  if (lane == 0) seg[wave] = s;
  __syncthreads();
  double z = 0.0;
  for (int i = 0; i < kRowWaves; ++i) z += seg[i];
  const int d = a.draft[(int64_t)b * a.k + slot];
  return (double)a.u_accept[(int64_t)b * a.k + slot] * z < weight64_full(logit<T>(row, d), m, inv);
}

// ---------------------------------------------------------------- kernels
// Small calls: one part of one row.
template <typename T>
__global__ __launch_bounds__(kPartThreads) void verify_part_kernel(VerifyArgs a) {
  const int part = (int)(blockIdx.x % a.parts);
  const int64_t rowid = blockIdx.x / a.parts;
  const int slot = (int)(rowid / a.B), b = (int)(rowid % a.B);
  if (slot > clamp_valid(a, b)) return;
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  const int j0 = part * a.part_size;
  const int j1 = a.V - j0 < a.part_size ? a.V : j0 + a.part_size;
  const VerifyPart p = row_stats<T, kPartThreads>(row_ptr(a, b, slot, T::kBytes), j0, j1, greedy,
                                                  greedy ? 1.f : inv_log2(temp));
  if (threadIdx.x == 0) a.part[((int64_t)b * (a.k + 1) + slot) * a.parts + part] = p;
}

// ---------------------------------------------------------------- phases of a large call
// Phase 0 is slot 0, 1: slots 1-2, 2: 3-6, 3: the rest.
constexpr int kPhases = 4;
__device__ __host__ __forceinline__ int phase_begin(int phase) {
  return phase == 0 ? 0 : (1 << phase) - 1;
}
__device__ __host__ __forceinline__ int phase_end(int phase, int k) {
  const int e = phase == kPhases - 1 ? k : (2 << phase) - 2;
  return e < k ? e : k;
}
__device__ __host__ __forceinline__ int last_phase(int k) {
  return k == 0 ? 0 : (k < 3 ? 1 : (k < 7 ? 2 : 3));
}
__device__ __forceinline__ int phase_of(int slot) {
  return slot == 0 ? 0 : (slot < 3 ? 1 : (slot < 7 ? 2 : 3));
}

// Logits of one of `parts` parts of a row.
__device__ __forceinline__ int phase_part(int V, int parts) {
  return ((V + parts - 1) / parts + 7) / 8 * 8;
}

// A row's parts, `parts` of them, as one; eight loads are in flight together.
__device__ __forceinline__ VerifyPart join_row(const VerifyArgs& a, int64_t row, int parts,
                                               float c) {
  const VerifyPart* p = a.part + row * a.parts;
  VerifyPart r{-__builtin_inff(), 0.f, 0x7fffffff, 0};
  for (int i = 0; i < parts; i += 8) {
    VerifyPart q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = p[i + k < parts ? i + k : i];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < parts) r = join(r, q[k], c);
  }
  return r;
}

// Slot 0: one workgroup per request.  stop[phase][b] is the lowest slot of request b that phase
// knows to be rejected; none yet (num_valid).
template <typename T>
__global__ __launch_bounds__(kRowThreads) void verify_first_kernel(VerifyArgs a) {
  const int b = blockIdx.x;
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  const VerifyPart p = row_stats<T, kRowThreads>(row_ptr(a, b, 0, T::kBytes), 0, a.V, greedy,
                                                 greedy ? 1.f : inv_log2(temp));
  if (threadIdx.x == 0) {
    a.part[(int64_t)b * (a.k + 1) * a.parts] = p;
    a.stop[b] = clamp_valid(a, b);
    if (b == 0) a.phase_parts[0] = 1;
  }
}

// A later phase.  Every workgroup first makes the tests of the phase before (a few loads a thread;
// joining the workgroups through memory instead took fences that cost more than the rows), which
// gives them all the same list of requests that are undecided, and then takes its share of the
// parts of their rows.
template <typename T>
__global__ __launch_bounds__(kPhaseThreads) void verify_phase_kernel(VerifyArgs a, int phase) {
  __shared__ int stop[kVerifyMaxOrdered], live[kVerifyMaxOrdered], count;
  const int tid = threadIdx.x, lane = tid & 63;
  for (int b = tid; b < a.B; b += kPhaseThreads) stop[b] = a.stop[(phase - 1) * a.B + b];
  __syncthreads();
  {
    const int q0 = phase_begin(phase - 1), q1 = phase_end(phase - 1, a.k);
    const int parts = a.phase_parts[phase - 1];
    const int groups = phase == 1 ? a.V / (8 * kRowThreads) + 1
                                  : phase_part(a.V, parts) / (8 * kPhaseThreads) + 1;
    for (int i = tid; i < a.B * (q1 - q0 + 1); i += kPhaseThreads) {
      const int b = i % a.B, slot = q0 + i / a.B;
      if (slot >= stop[b]) continue;  // not read, known, or past the draft
      const float temp = temperature(a, b);
      const bool greedy = !(temp > 0.f);
      const float c = greedy ? 1.f : inv_log2(temp);
      const VerifyPart p = join_row(a, (int64_t)b * (a.k + 1) + slot, parts, c);
      if (test_slot<T>(a, b, slot, p, greedy, c, groups) == kReject) atomicMin(&stop[b], slot);
    }
  }
  __syncthreads();
  const int s0 = phase_begin(phase), s1 = phase_end(phase, a.k);
  if (tid < 64) {
    int n = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
      const int b = b0 + lane;
      const bool in = b < a.B && stop[b] >= s0;
      const unsigned long long any = __ballot(in);
      if (in) live[n + __popcll(any & ((1ull << lane) - 1))] = b;
      n += __popcll(any);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n = count;
  // The number of parts that makes the busiest workgroup's time least: its rounds, each a part of
  // a row and about 1/8 of one besides (starting the loads, joining the threads).
  const int64_t rows = (int64_t)n * (s1 - s0 + 1);
  int parts = 1;
  float least = 3.4e38f;
  for (int p = 1; p <= a.parts && p * 4096 <= a.V; ++p) {
    const float t = (float)((rows * p + kPhaseGroups - 1) / kPhaseGroups) * (1.f / p + 0.125f);
    if (t < least) {
      least = t;
      parts = p;
    }
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.B; b += kPhaseThreads) a.stop[phase * a.B + b] = stop[b];
    if (tid == 0) a.phase_parts[phase] = parts;
  }
  const int size = phase_part(a.V, parts);
  for (int64_t i = blockIdx.x; i < rows * parts; i += gridDim.x) {
    const int part = (int)(i % parts);
    const int64_t r = i / parts;
    const int slot = s0 + (int)(r / n), b = live[r % n];
    if (slot > stop[b]) continue;  // past num_valid
    const float temp = temperature(a, b);
    const bool greedy = !(temp > 0.f);
    const int j0 = part * size < a.V ? part * size : a.V;
    const int j1 = a.V - j0 < size ? a.V : j0 + size;
    const VerifyPart p = row_stats<T, kPhaseThreads>(row_ptr(a, b, slot, T::kBytes), j0, j1,
                                                     greedy, greedy ? 1.f : inv_log2(temp));
    if (tid == 0) a.part[((int64_t)b * (a.k + 1) + slot) * a.parts + part] = p;
  }
}

// What a request's draw starts from: the number accepted and the row's statistics.
struct Drawn {
  int n;
  float m;
  int at;
};

// kSmall: the rows' statistics are made here, a wavefront a row; otherwise they have been stored.
template <typename T, bool kSmall>
__device__ Drawn accepted(const VerifyArgs& a, int b, float temp, bool greedy, double* seg,
                          const double* table) {
  __shared__ float row_m[kMaxRows];
  __shared__ int row_at[kMaxRows], verdict[kMaxRows];
  // rows past `end` have no statistics; slot `end` is past the draft or known to be rejected
  const int tid = threadIdx.x;
  const int end = !kSmall && a.stop ? a.stop[last_phase(a.k) * a.B + b] : clamp_valid(a, b);
  const float c = greedy ? 1.f : inv_log2(temp);
  if constexpr (kSmall) {
    __shared__ VerifyPart own[kMaxRows];
    const int lane = tid & 63;
    for (int slot = tid >> 6; slot <= end; slot += kRowWaves) {
      const char* row = row_ptr(a, b, slot, T::kBytes);
      VerifyPart r = wave_stats<T, 1, false>(row, lane * 8, a.V, 512, greedy, c);
      if (to_clean(r)) r = wave_stats<T, 1, true>(row, lane * 8, a.V, 512, greedy, c);
      if (lane == 0) own[slot] = r;
    }
    __syncthreads();
    if (tid <= end) {
      row_m[tid] = own[tid].m;
      row_at[tid] = own[tid].at;
      verdict[tid] = tid < end ? test_slot<T>(a, b, tid, own[tid], greedy, c, a.V / 512 + 1)
                               : kReject;
    }
  } else if (tid <= end) {
    const int64_t row = (int64_t)b * (a.k + 1) + tid;
    const int phase = phase_of(tid);
    const int parts = a.stop ? a.phase_parts[phase] : a.parts;
    const VerifyPart r = join_row(a, row, parts, c);
    const int groups = 1 + (!a.stop ? a.part_size / (8 * kPartThreads)
                                    : phase == 0 ? a.V / (8 * kRowThreads)
                                                 : phase_part(a.V, parts) / (8 * kPhaseThreads));
    row_m[tid] = r.m;
    row_at[tid] = r.at;
    verdict[tid] = tid < end ? test_slot<T>(a, b, tid, r, greedy, c, groups) : kReject;
  }
  __syncthreads();
  int n = 0;
  for (; n < end; ++n) {
    bool ok = verdict[n] == kAccept;
    if (verdict[n] == kClose)
      ok = test_close<T>(a, b, n, weights64(table, row_m[n], temp, greedy), row_m[n],
                         inv64(temp), seg);
    if (!ok) break;
  }
  return Drawn{n, row_m[n], row_at[n]};
}

// One value a thread, in order: the first thread whose running sum (from `base`) passes t, or the
// last that holds anything where rounding hides that one; -1 when all are nothing.  `before`: the
// sum ahead of it; with `fresh`, t is first set to u times the whole sum.
struct Found {
  int at;
  double before, t;
};
__device__ Found find_in_block(double x, double least, double base, double t, bool fresh, double u,
                               double* seg) {
  __shared__ int found;
  __shared__ double found_before;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  double inc = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(inc, o);
    if (lane >= o) inc += y;
  }
  double exc = __shfl_up(inc, 1);
  if (lane == 0) exc = 0.0;
  __syncthreads();
  if (lane == 63) seg[wave] = inc;
  if (tid == 0) found = 0x7fffffff;
  __syncthreads();
  double before = base, z = 0.0;
  for (int i = 0; i < kRowWaves; ++i) {
    if (i < wave) before += seg[i];
    z += seg[i];
  }
  if (fresh) t = u * z;
  const unsigned long long some = __ballot(x > least);
  const unsigned long long hit = __ballot(x > least && before + inc > t);
  if (hit && lane == 0) atomicMin(&found, tid + __ffsll((long long)hit) - 1);
  __syncthreads();
  const bool hidden = found == 0x7fffffff;
  __syncthreads();
  if (hidden) {
    if (tid == 0) found = -1;
    __syncthreads();
    if (some && lane == 0) atomicMax(&found, tid + 63 - __clzll(some));
    __syncthreads();
  }
  const int at = found;
  if (tid == at) found_before = before + exc;
  __syncthreads();
  const double ahead = at >= 0 ? found_before : base;
  __syncthreads();
  return Found{at, ahead, t};
}

// Few requests over a large vocabulary: the fp64 sums of a request's row, `pieces` workgroups of
// kRowWaves segments each.  Every one makes the request's tests again; the first stores their
// outcome.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void verify_sums_kernel(VerifyArgs a) {
  __shared__ double seg[kRowWaves], table[kTable];
  const int b = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  fill_table(table);
  __syncthreads();
  const Drawn r = accepted<T, false>(a, b, temp, greedy, seg, table);
  if (piece == 0 && threadIdx.x == 0) a.outcome[b] = VerifyPart{r.m, 0.f, r.at, r.n};
  if (greedy || !(r.m > -__builtin_inff())) return;
  const int d = r.n < clamp_valid(a, b) ? a.draft[(int64_t)b * a.k + r.n] : -1;
  const int j0 = seg_at(0, a.V, piece, a.pieces), j1 = seg_at(0, a.V, piece + 1, a.pieces);
  const double s = wave_range64<T>(row_ptr(a, b, r.n, T::kBytes), seg_at(j0, j1, wave, kRowWaves),
                                   seg_at(j0, j1, wave + 1, kRowWaves),
                                   weights64(table, r.m, temp, false), d, lane);
  if (lane == 0) a.sums[((int64_t)b * a.pieces + piece) * kRowWaves + wave] = s;
}

// One workgroup per request: the tests in order (of a large call those of its last phase and any
// too close for fp32), then the draw from the row they end at.  The row is summed in segments, the
// segment that holds the draw in turn, until 1024 logits are left, which are taken one a thread.
template <typename T, bool kSmall>
__global__ __launch_bounds__(kRowThreads) void verify_draw_kernel(VerifyArgs a) {
  __shared__ double seg[kRowWaves], table[kTable];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float temp = temperature(a, b);
  const bool greedy = !(temp > 0.f);
  Drawn r;
  if (!kSmall && a.pieces > 1) {
    const VerifyPart p = a.outcome[b];
    r = Drawn{p.pad, p.m, p.at};
  } else {
    fill_table(table);
    __syncthreads();
    r = accepted<T, kSmall>(a, b, temp, greedy, seg, table);
  }
  int pick = -1;
  if (r.m > -__builtin_inff()) {
    pick = r.at;
    if (!greedy) {
      const int d = r.n < clamp_valid(a, b) ? a.draft[(int64_t)b * a.k + r.n] : -1;
      const char* row = row_ptr(a, b, r.n, T::kBytes);
      const double u = a.u_sample[b], inv = inv64(temp);
      int j0 = 0, j1 = a.V;
      double base = 0.0, t = 0.0;
      bool fresh = true, none = false;
      if (!kSmall && a.pieces > 1) {
        const int segs = a.pieces * kRowWaves;
        const double x = tid < segs ? a.sums[(int64_t)b * segs + tid] : 0.0;
        const Found f = find_in_block(x, kTiny, base, t, fresh, u, seg);
        none = f.at < 0;
        const int s = f.at < 0 ? 0 : f.at;
        const int p0 = seg_at(0, a.V, s / kRowWaves, a.pieces);
        const int p1 = seg_at(0, a.V, s / kRowWaves + 1, a.pieces);
        j0 = seg_at(p0, p1, s % kRowWaves, kRowWaves);
        j1 = seg_at(p0, p1, s % kRowWaves + 1, kRowWaves);
        base = f.before;
        t = f.t;
        fresh = false;
        if (j1 - j0 > kRowThreads) {
          fill_table(table);
          __syncthreads();
        }
      }
      while (j1 - j0 > kRowThreads) {
        const Weights64 w = weights64(table, r.m, temp, false);
        const double s = wave_range64<T>(row, seg_at(j0, j1, wave, kRowWaves),
                                         seg_at(j0, j1, wave + 1, kRowWaves), w, d, lane);
        __syncthreads();
        if (lane == 0) seg[wave] = s;
        __syncthreads();
        if (fresh) {
          double z = 0.0;
          for (int i = 0; i < kRowWaves; ++i) z += seg[i];
          t = u * z;
          none = !(z > kTiny);
          fresh = false;
        }
        // the segment whose sums pass t; the last that holds anything if rounding hides it
        int at = 0;
        double before = base, run = base;
        for (int i = 0; i < kRowWaves; ++i)
          if (seg[i] > kTiny) {
            at = i;
            before = run;
            run += seg[i];
            if (run > t) break;
          }
        base = before;
        const int s0 = seg_at(j0, j1, at, kRowWaves), s1 = seg_at(j0, j1, at + 1, kRowWaves);
        j0 = s0;
        j1 = s1;
      }
      const bool tiny = !fresh && t < kTiny;
      if (!none && !tiny) {
        const int j = j0 + tid;
        double x = 0.0;
        if (j < j1 && j != d) x = weight64_full(logit<T>(row, j), r.m, inv);
        const int at = find_in_block(x, 0.0, base, t, fresh, u, seg).at;
        if (at >= 0) pick = j0 + at;
      } else if (!none) {
        // A draw this close to 0 can land on weights that the fast ones leave out.
        __shared__ int found;
        if (wave == 0) {
          double run = 0.0;
          int last = -1;
          for (int i = 0; i < a.V; i += 64) {
            double y = 0.0;
            if (i + lane < a.V && i + lane != d)
              y = weight64_full(logit<T>(row, i + lane), r.m, inv);
            double sum = y;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
              const double v = __shfl_up(sum, o);
              if (lane >= o) sum += v;
            }
            const unsigned long long h = __ballot(y > 0.0 && run + sum > t);
            if (h) {
              last = i + __ffsll((long long)h) - 1;
              break;
            }
            run += __shfl(sum, 63);
          }
          if (lane == 0) found = last;
        }
        __syncthreads();
        if (found >= 0) pick = found;
      }
    }
  }
  if (tid <= a.k)
    a.sampled[(int64_t)b * (a.k + 1) + tid] =
        tid < r.n ? a.draft[(int64_t)b * a.k + tid] : (tid == r.n ? pick : -1);
  if (tid == 0) a.num_accepted[b] = r.n;
}

template <typename T>
hipError_t launch_type(const VerifyArgs& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.B * (a.k + 1);
  const dim3 requests((unsigned)a.B), whole(kRowThreads);
  if (a.small) {
    hipLaunchKernelGGL((verify_draw_kernel<T, true>), requests, whole, 0, st, a);
    return hipGetLastError();
  }
  if (a.stop) {
    hipLaunchKernelGGL(verify_first_kernel<T>, requests, whole, 0, st, a);
    for (int phase = 1; phase <= last_phase(a.k); ++phase)
      hipLaunchKernelGGL(verify_phase_kernel<T>, dim3(kPhaseGroups), dim3(kPhaseThreads), 0, st, a,
                         phase);
  } else {
    hipLaunchKernelGGL(verify_part_kernel<T>, dim3((unsigned)(rows * a.parts)),
                       dim3(kPartThreads), 0, st, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.pieces > 1) {
    hipLaunchKernelGGL(verify_sums_kernel<T>, dim3((unsigned)(a.B * a.pieces)), whole, 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((verify_draw_kernel<T, false>), requests, whole, 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t verify_plan(VerifyArgs* a, KvType type) {
  const int bytes = type == kFp32 ? 4 : 2;
  const int64_t rows = (int64_t)a->B * (a->k + 1);
  a->in_order = false;
  a->parts = a->pieces = 1;
  a->part_size = a->V;
  a->small = a->V <= kSmallV;
  if (a->small) return 0;
  // Phases pay from about 0.4 GB of logits: at B = 256, k = 32, V = 32000 (0.54 GB) 90 us against
  // 145 when 64% of the drafted tokens are accepted, 220 against 143 when all are; at 1.3 GB 154
  // against 298 and 367 against 297; at 0.28 GB 86 against 81 and 148 against 82.
  a->in_order = a->B <= kVerifyMaxOrdered && (double)rows * a->V * bytes >= 4e8;
  if (a->in_order) {
    a->parts = kVerifyMaxParts;
  } else {
    // parts of at least 16K logits, enough of them to fill 256 CUs four times over
    int64_t parts = rows > 0 ? (1024 + rows - 1) / rows : 1;
    const int64_t most = ((int64_t)a->V + 16383) / 16384;
    parts = parts > most ? most : parts;
    parts = parts < 1 ? 1 : parts;
    const int64_t size = (a->V + parts - 1) / parts;
    a->part_size = (int32_t)((size + 7) / 8 * 8);
    a->parts = (int32_t)((a->V + a->part_size - 1) / a->part_size);
  }
  // the drawn rows' fp64 sums: one workgroup per CU, of at least 4K logits, 1024 segments a row
  int64_t pieces = a->B > 0 ? 256 / a->B : 1;
  pieces = pieces > a->V / 4096 ? a->V / 4096 : pieces;
  pieces = pieces > kRowThreads / kRowWaves ? kRowThreads / kRowWaves : pieces;
  a->pieces = pieces < 1 ? 1 : (int32_t)pieces;
  size_t size = (size_t)rows * a->parts * sizeof(VerifyPart);
  if (a->pieces > 1)
    size += (size_t)a->B * (sizeof(VerifyPart) + a->pieces * kRowWaves * sizeof(double));
  if (a->in_order) size += (size_t)kPhases * (a->B + 1) * sizeof(int32_t);
  return size;
}

int64_t verify_threads(const VerifyArgs& a) {
  const int64_t draws = (int64_t)a.B * a.pieces * kRowThreads;
  if (a.small || a.in_order) return draws;
  const int64_t parts = (int64_t)a.B * (a.k + 1) * a.parts * kPartThreads;
  return parts > draws ? parts : draws;
}

void verify_place(VerifyArgs* a, void* workspace) {
  const size_t rows = (size_t)a->B * (a->k + 1);
  a->part = (VerifyPart*)workspace;
  VerifyPart* next = a->part + rows * a->parts;
  a->outcome = nullptr;
  a->sums = nullptr;
  if (a->pieces > 1) {
    a->outcome = next;
    a->sums = (double*)(a->outcome + a->B);
    next = (VerifyPart*)(a->sums + (size_t)a->B * a->pieces * kRowWaves);
  }
  a->stop = a->in_order ? (int32_t*)next : nullptr;
  a->phase_parts = a->in_order ? a->stop + (size_t)kPhases * a->B : nullptr;
}

hipError_t launch_verify(const VerifyArgs& a, KvType type, hipStream_t st) {
  if (a.B <= 0) return hipSuccess;
  if (type == kBf16) return launch_type<Bf16>(a, st);
  if (type == kFp16) return launch_type<Fp16>(a, st);
  return launch_type<Fp32>(a, st);
}

}  // namespace sfx

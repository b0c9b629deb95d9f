// pages.hip -- pages handed out and taken back on the device, and the layout of a packed batch.
//
// Reserve.  Request b holds held[b] pages (the first entries of its table row) and needs
// ceil(tokens[b] / page_size).  Pages it no longer needs are released, in order of (request,
// entry); R of them in all.  Requests that need more get all or nothing, in order: request b is
// served when the running sum W(b) of what is wanted up to it stays within num_free + R.  As W
// does not fall, the served ones are those up to some request, and A = the largest W(b) within the
// limit is what they take.  Page number a of these is the a-th released one, and from a = R on
// free_pages[num_free - 1 - (a - R)]; released pages past the A-th go behind the free list.  So every
// page that moves is one item x < max(R, A) with one source and one destination, found by binary
// search in the running sums; nothing depends on the order in which items run.
//
// Measured: 32 requests 4.1 us, bounded by dependent steps of one workgroup; 1024 requests of which a
// quarter ends and another comes in (some 60000 pages move) 4.6 us for the sums and 5.3 for the
// moves.
//
// Layout.  offsets = running sum of the counts.  Every workgroup makes the whole sum for itself (it
// reads B counts from L2, which costs less than a launch) and looks its own rows up in it.  Measured:
// 64 requests of 17 rows 3.4 us, 256 requests of 20000 rows 4.3 us.
#include "pages.h"

namespace sfx {

namespace {

constexpr int kThreads = 1024, kWaveCount = kThreads / 64;
// Requests whose running sums one workgroup keeps in LDS.
constexpr int kLdsRequests = 4096;
// Table entries up to which one workgroup moves all pages itself.  With a quarter of the requests
// ending and another coming in, a call of 33000 entries takes 8.4 us so and 12.3 in two launches, one
// of 65000 14.7 and 12.1, one of 540000 81 and 12.2.
constexpr int64_t kOneGroupEntries = 40960;

// Inclusive running sum over the workgroup; `total` receives the whole.  Sums stay below 2^31.
__device__ __forceinline__ int scan(int x, int* waves, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // of the last use of `waves`
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaveCount; ++w) {
    const int y = waves[w];
    before += w < wave ? y : 0;
    all += y;
  }
  total = all;
  return x + before;
}

// Least i with sums[i] > x; sums does not fall and its last entry passes x.
__device__ __forceinline__ int find(const int* sums, int n, int x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    lo = sums[lo + half - 1] > x ? lo : lo + half;
    n -= half;
  }
  return lo;
}

// What request b holds, would hold and wants.
struct Need {
  int held, back, want;  // back: pages released, want: pages wanted where they can fit at all
  int miss;              // pages wanted in any case
};
__device__ __forceinline__ Need need_of(const ReserveArgs& a, int b) {
  Need n{0, 0, 0, 0};
  if (b >= a.B) return n;
  const int t = a.tokens[b], h = a.held[b];
  const int need = t > 0 ? (t - 1) / a.page_size + 1 : 0;
  n.held = h < 0 ? 0 : (h > a.max_pages ? a.max_pages : h);
  n.back = n.held > need ? n.held - need : 0;
  n.miss = need > n.held ? need - n.held : 0;
  n.want = need > a.max_pages ? 0 : n.miss;
  return n;
}

struct Totals {
  int released, granted, num_free;
};

// Moves page number x of the call.
__device__ __forceinline__ void move(const ReserveArgs& a, const Totals& t, const int* back,
                                     const int* want, const int* held, int x) {
  int page;
  if (x < t.released) {
    const int b = find(back, a.B, x);
    // request b's released entries are the last back[b] - back[b - 1] of the held ones
    const int64_t at = (int64_t)b * a.max_pages + held[b] - (back[b] - x);
    page = a.page_table[at];
    a.page_table[at] = -1;
  } else {
    page = a.free_pages[t.num_free - 1 - (x - t.released)];
  }
  if (x < t.granted) {
    const int b = find(want, a.B, x);
    a.page_table[(int64_t)b * a.max_pages + held[b] + x - (b ? want[b - 1] : 0)] = page;
  } else {
    const int64_t to = (int64_t)t.num_free + x - t.granted;
    if (to < a.num_pages) a.free_pages[to] = page;  // else: more pages than there are
  }
}

// The running sums `back` and `want` and the old `held`, and with them the new held, num_free and
// missing.
__device__ Totals plan(const ReserveArgs& a, int* back, int* want, int* held, int* waves) {
  int released = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const Need n = need_of(a, b);
    int total;
    const int sum = scan(n.back, waves, total) + released;
    released += total;
    if (b < a.B) {
      back[b] = sum;
      held[b] = n.held;
    }
  }
  Totals t{released, 0, *a.num_free};
  t.num_free = t.num_free < 0 ? 0 : (t.num_free > a.num_pages ? a.num_pages : t.num_free);
  const int64_t room = (int64_t)t.num_free + released;
  int wanted = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const Need n = need_of(a, b);  // of a request of this thread: not yet changed
    int total;
    const int sum = scan(n.want, waves, total) + wanted;
    wanted += total;
    const bool granted = n.want == n.miss && sum <= room;
    if (b < a.B) {
      want[b] = sum;
      a.held[b] = n.held - n.back + (granted ? n.want : 0);
      if (a.missing) a.missing[b] = granted ? 0 : n.miss;
    }
    // the largest sum within the room, over the workgroup: sums do not fall, so it is the sum
    // of the wants of the requests within it
    int part = b < a.B && sum <= room ? n.want : 0;
    scan(part, waves, total);
    t.granted += total;
  }
  __syncthreads();  // every thread has read num_free
  if (threadIdx.x == 0) {
    const int64_t left = room - t.granted;
    *a.num_free = left < a.num_pages ? (int)left : a.num_pages;
  }
  __syncthreads();
  return t;
}

// Everything in one workgroup.
__global__ __launch_bounds__(kThreads) void reserve_kernel(ReserveArgs a) {
  __shared__ int back[kLdsRequests], want[kLdsRequests], held[kLdsRequests], waves[kWaveCount];
  const Totals t = plan(a, back, want, held, waves);
  const int items = t.released > t.granted ? t.released : t.granted;
  for (int x = threadIdx.x; x < items; x += kThreads) move(a, t, back, want, held, x);
}

// The same in two launches: the sums into the workspace, then the pages by the whole card.
__global__ __launch_bounds__(kThreads) void reserve_plan_kernel(ReserveArgs a) {
  __shared__ int waves[kWaveCount];
  int* p = a.plan + 4;
  const Totals t = plan(a, p, p + a.B, p + 2 * (int64_t)a.B, waves);
  if (threadIdx.x == 0) {
    a.plan[0] = t.released;
    a.plan[1] = t.granted;
    a.plan[2] = t.num_free;
  }
}
// The sums are searched in LDS where they fit: 20 dependent reads from L2 would take 6 us.
__global__ __launch_bounds__(256) void reserve_move_kernel(ReserveArgs a) {
  __shared__ int sums[2][kLdsRequests];
  const int* back = a.plan + 4;
  const int* want = back + a.B;
  const Totals t{a.plan[0], a.plan[1], a.plan[2]};
  const int items = t.released > t.granted ? t.released : t.granted;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (first - threadIdx.x >= items) return;
  if (a.B <= kLdsRequests) {
    for (int b = threadIdx.x; b < a.B; b += 256) {
      sums[0][b] = back[b];
      sums[1][b] = want[b];
    }
    __syncthreads();
    for (int64_t x = first; x < items; x += (int64_t)gridDim.x * 256)
      move(a, t, sums[0], sums[1], want + a.B, (int)x);
  } else {
    for (int64_t x = first; x < items; x += (int64_t)gridDim.x * 256)
      move(a, t, back, want, want + a.B, (int)x);
  }
}

unsigned move_groups(int32_t B, int32_t max_pages) {
  const int64_t n = ((int64_t)B * max_pages + 255) / 256;
  return (unsigned)(n < 512 ? n : 512);
}

bool one_group(int32_t B, int32_t max_pages) {
  return B <= kLdsRequests && (int64_t)B * max_pages <= kOneGroupEntries;
}

__global__ __launch_bounds__(kThreads) void layout_kernel(LayoutArgs a) {
  __shared__ int sums[kThreads], waves[kWaveCount];
  // thread i sums requests i per .. (i + 1) per - 1
  const int per = (a.B + kThreads - 1) / kThreads;
  const int first = threadIdx.x * per;
  // a count as it is used: not below 0, not past the largest position, N at most
  auto count_of = [&](int b, int& start) {
    start = a.start[b];
    start = start < 0 ? 0 : start;
    int c = a.count[b];
    c = c < 0 ? 0 : (c > a.N ? a.N : c);
    return c > 0x7fffffff - start ? 0x7fffffff - start : c;
  };
  // sums are cut at N, so that no sum of two passes 2^32
  auto add = [&](unsigned x, unsigned y) {
    const unsigned s = x + y;
    return s > (unsigned)a.N ? (unsigned)a.N : s;
  };
  unsigned mine = 0;
  for (int b = first; b < first + per && b < a.B; ++b) {
    int start;
    mine = add(mine, count_of(b, start));
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  unsigned x = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned y = __shfl_up(x, o);
    if (lane >= o) x = add(x, y);
  }
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  unsigned before = 0;
  for (int w = 0; w < wave; ++w) before = add(before, waves[w]);
  x = add(x, before);
  sums[threadIdx.x] = x;
  const unsigned prev = __shfl_up(x, 1);
  __syncthreads();
  unsigned at = threadIdx.x == 0 ? 0 : (lane == 0 ? sums[threadIdx.x - 1] : prev);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.offsets[0] = 0;
    for (int b = first; b < first + per && b < a.B; ++b) {
      int start;
      const unsigned end = add(at, count_of(b, start));
      a.offsets[b + 1] = end;
      if (a.seq_lens) a.seq_lens[b] = start + (int)(end - at);
      at = end;
    }
  }
  if (!a.request && !a.position && !a.slots) return;
  const int64_t row = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (row >= a.N) return;
  int b = -1, pos = -1;
  int64_t slot = -1;
  if (row < sums[kThreads - 1]) {
    const int seg = find(sums, kThreads, (int)row);
    unsigned from = seg ? sums[seg - 1] : 0;
    b = seg * per;
    int start;
    for (;; ++b) {  // ends: the segment's sum passes the row
      const unsigned end = add(from, count_of(b, start));
      if (end > row) break;
      from = end;
    }
    pos = start + (int)(row - from);
    const int pi = pos / a.page_size;
    if (a.slots && pi < a.max_pages) {  // there may be no table for the others
      const int page = a.page_table[(int64_t)b * a.max_pages + pi];
      if (page >= 0 && page < a.num_pages) slot = (int64_t)page * a.page_size + pos % a.page_size;
    }
  }
  if (a.request) a.request[row] = b;
  if (a.position) a.position[row] = pos;
  if (a.slots) a.slots[row] = slot;
}

unsigned layout_groups(int32_t N) { return N > 0 ? (unsigned)(((int64_t)N + kThreads - 1) / kThreads) : 1; }

}  // namespace

size_t reserve_plan_words(int32_t B, int32_t max_pages) {
  return one_group(B, max_pages) ? 0 : 4 + 3 * (size_t)B;
}

int64_t layout_threads(int32_t N) { return (int64_t)layout_groups(N) * kThreads; }

hipError_t launch_reserve(const ReserveArgs& a, hipStream_t st) {
  if (one_group(a.B, a.max_pages)) {
    hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(reserve_plan_kernel, dim3(1), dim3(kThreads), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.max_pages == 0) return hipSuccess;
  hipLaunchKernelGGL(reserve_move_kernel, dim3(move_groups(a.B, a.max_pages)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_layout(const LayoutArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(layout_kernel, dim3(layout_groups(a.N)), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace sfx

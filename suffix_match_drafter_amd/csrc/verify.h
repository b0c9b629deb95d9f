// verify.h -- launch interface of the draft verification (internal to libsfx).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_cache.h"

namespace sfx {

// What one workgroup saw of its part of a row (or of all of it).
struct VerifyPart {
  float m;     // largest logit (-inf: none)
  float s;     // sum of 2^((l - m) / (T ln 2))
  int32_t at;  // lowest index of the largest
  int32_t pad;
};

struct VerifyArgs {
  int32_t B, k, V;
  const void* logits;
  int64_t batch_stride, slot_stride;  // elements
  const float* temperature;           // NULL: 1
  const int32_t* draft;
  const int32_t* num_valid;
  const float* u_accept;
  const float* u_sample;
  int32_t* sampled;
  int32_t* num_accepted;
  // plan (verify_plan)
  bool small;         // one launch: a workgroup makes its request's statistics itself
  bool in_order;      // slots in phases, rows past a rejection left out
  int32_t parts;      // parts of one row (in_order: the most)
  int32_t part_size;  // its logits (not in_order)
  VerifyPart* part;   // [B][k + 1][parts]
  int32_t* stop;      // [phases][B] lowest slot known to be rejected (in_order, else NULL)
  int32_t* phase_parts;  // [phases] parts of a row (in_order, else NULL)
  int32_t pieces;        // workgroups over the fp64 sums of a drawn row
  VerifyPart* outcome;   // [B] m and at of the row drawn from, pad = its slot (pieces > 1)
  double* sums;          // [B][pieces][16] (pieces > 1)
};

constexpr int kVerifyMaxParts = 16;      // of a row, in_order
constexpr int kVerifyMaxOrdered = 2048;  // requests of an in_order call (a list in LDS)

// Fills the plan from the shapes; returns the workspace bytes it needs.
size_t verify_plan(VerifyArgs* a, KvType type);

// Threads of the largest of the planned launches.
int64_t verify_threads(const VerifyArgs& a);

// Places the plan's buffers in the workspace.
void verify_place(VerifyArgs* a, void* workspace);

hipError_t launch_verify(const VerifyArgs& a, KvType type, hipStream_t st);

}  // namespace sfx

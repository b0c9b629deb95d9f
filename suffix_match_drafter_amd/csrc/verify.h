// verify.h -- launch interface of the draft verification (internal to libsfx).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_cache.h"

namespace sfx {

// What one workgroup saw of its part of a row.
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
  // plan
  int32_t parts;      // workgroups of one row
  int32_t part_size;  // its logits
  VerifyPart* part;   // [B][k + 1][parts]
};

size_t verify_plan(VerifyArgs* a);
hipError_t launch_verify(const VerifyArgs& a, KvType type, hipStream_t st);

}  // namespace sfx

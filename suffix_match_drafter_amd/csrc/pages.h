// pages.h -- launch interface of the page allocation and the packed batch's layout (internal to
// libsfx).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfx {

struct ReserveArgs {
  int32_t B, max_pages, page_size, num_pages;
  const int32_t* tokens;
  int32_t* page_table;
  int32_t* held;
  int32_t* free_pages;
  int32_t* num_free;
  int32_t* missing;  // NULL: not wanted
  int32_t* plan;     // workspace of calls in two launches: reserve_plan_words words
};

// Words of workspace: 0 for calls that one workgroup does.
size_t reserve_plan_words(int32_t B, int32_t max_pages);

struct LayoutArgs {
  int32_t B, N, max_pages, page_size, num_pages;
  const int32_t* page_table;
  const int32_t* start;
  const int32_t* count;
  int32_t* offsets;
  int32_t* seq_lens;  // these four may be NULL
  int32_t* request;
  int32_t* position;
  int64_t* slots;
};
int64_t layout_threads(int32_t N);

hipError_t launch_reserve(const ReserveArgs& a, hipStream_t st);
hipError_t launch_layout(const LayoutArgs& a, hipStream_t st);

}  // namespace sfx

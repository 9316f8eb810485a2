// Eviction from a paged cache by accumulated attention weight: arguments.
#pragma once

#include "ds4a_internal.cuh"

namespace ds4a {

struct EvictArgs {
  int B, m, budget, recent, cap;
  uint8_t* pages;
  int row_bytes, n_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* q_pos;
  const uint16_t* w;  // nullable
  int64_t w_stride;
  float* acc;
  int32_t* entry;
  int64_t stride;  // of acc and entry
  int32_t* drop;
  int32_t* moves;  // [B]
  int32_t* list;   // [B][2][budget]: destination and source slots
  unsigned int* err;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

}  // namespace ds4a

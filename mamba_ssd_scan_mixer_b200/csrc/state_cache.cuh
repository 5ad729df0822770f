// The 8-bit state cache: problem description.
#pragma once

#include "common.cuh"

namespace m2 {

struct StateCacheArgs {
  int64_t batch, n, nslots;
  int block, format, state_dtype;
  void *state;  // working states, row stride ld
  int64_t ld;
  const int32_t *slots;
  void *codes;      // [nslots, n]
  uint8_t *scales;  // [nslots, ceil(n / block)]
  cudaStream_t stream;
};

cudaError_t state_cache_store(const StateCacheArgs &a);
cudaError_t state_cache_load(const StateCacheArgs &a);
cudaError_t take_state_cache_errors(unsigned int *out);

}  // namespace m2

// The expert-sorted row layout; see expert_map.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct ExpertMapParams {
  const int32_t* ids;
  int32_t* row_map;  // null: not wanted
  int32_t* row_token;
  int32_t* offsets;
  int32_t* counts;
  int64_t n_rows;
  int64_t slots;  // T * k
  int E, k, block;
  int rest;           // 1: slots whose id is outside [0, E - 1) go to group E - 1
  int32_t* err_flag;  // with rest: MOE_FLAG_BAD_INDEX for an id above E - 2
};

cudaError_t launch_expert_map(const ExpertMapParams& p, cudaStream_t stream);

}  // namespace moe

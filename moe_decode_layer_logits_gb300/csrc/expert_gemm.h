// Tensor-core products of row segments with their weights; see expert_gemm.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct ExpertGemm {
  const void* x;             // [n_x, K] BF16
  const int32_t* row_token;  // [n_rows] or null
  const void* w;             // [E, N, K] BF16
  const int32_t* offsets;    // [E], null: one segment of all rows (E = 1)
  const int32_t* counts;     // [E]
  void* out;                 // [n_rows, N or N/2] BF16
  int64_t n_x, n_rows, E, N, K;
  bool swiglu;
  float* partial;  // workspace of expert_gemm_workspace() bytes
  int32_t* err_flag;
};

// Bytes of the FP32 partial tiles.
int64_t expert_gemm_workspace(int64_t n_rows);

cudaError_t launch_expert_gemm(const ExpertGemm& g, cudaStream_t stream);

}  // namespace moe

// Tensor-core products of row segments with their weights; see expert_gemm.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct ExpertGemm {
  const void* x;             // [n_x, K] BF16
  const int32_t* row_token;  // [n_rows] or null
  const void* w;             // [E, N, K] BF16
  const int32_t* offsets;    // [E]
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

// Test hook of the bounded waits: the stage that the next call's product
// launches withhold, or -1; taking it clears it.
int take_withheld_stage();

// MOE_OK if N, K and act are sizes that the products take.
int check_linear(int64_t N, int64_t K, int32_t act);

struct AdapterLinear {
  const uint16_t* x;    // [T, K]
  const uint16_t* w;    // [N, K]
  const uint16_t* a;    // [L, R, K]
  const uint16_t* b;    // [L, N, R]
  const int32_t* ids;   // [T]
  const float* scale;   // [L]
  uint16_t* out;        // [T, N or N/2]
  int64_t T, N, K;
  int R, L;
  bool swiglu;
  uint8_t* workspace;  // adapter_workspace() bytes
  int32_t* err_flag;
};

int64_t adapter_workspace(int64_t T, int64_t N, int64_t K, int R, int L);

cudaError_t launch_adapter_linear(const AdapterLinear& g, cudaStream_t stream);

}  // namespace moe

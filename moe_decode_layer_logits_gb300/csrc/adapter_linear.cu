// moe_adapter_linear: argument checks; the kernels are in adapter_gemm.cu.
#include "expert_gemm.h"
#include "host_util.h"

extern "C" int64_t moe_adapter_linear_workspace(int64_t T, int64_t N, int64_t K, int32_t R, int32_t L) {
  if (T < 0 || N < 1 || K < 1 || R < 1 || L < 1 || T > 0x7FFFFFFFll / R || N > MOE_MAX_DIM || L > MOE_MAX_ADAPTERS)
    return -1;
  return T == 0 ? 0 : moe::adapter_workspace(T, N, K, R, L);
}

extern "C" int moe_adapter_linear(const void* x_bf16, const void* w_bf16, const void* adapter_a_bf16,
                                  const void* adapter_b_bf16, const int32_t* adapter_ids,
                                  const float* adapter_scale, void* out_bf16, int64_t T, int64_t N, int64_t K,
                                  int32_t R, int32_t L, int32_t act, void* workspace, int64_t workspace_bytes,
                                  int32_t* err_flag, cudaStream_t stream) {
  using namespace moe;
  if (T < 0 || R < 1 || L < 1 || workspace_bytes < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(N, K, act);
  if (st != MOE_OK) return st;
  if (R % 8 != 0 || R > MOE_MAX_RANK || L > MOE_MAX_ADAPTERS || T > 0x7FFFFFFFll / R) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !w_bf16 || !adapter_a_bf16 || !adapter_b_bf16 || !adapter_ids || !adapter_scale || !out_bf16)
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_adapter_linear_workspace(T, N, K, R, L) || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(adapter_a_bf16, 16) || !aligned(adapter_b_bf16, 16) ||
      !aligned(out_bf16, 16) || !aligned(workspace, 16) || !aligned(adapter_ids, 4) || !aligned(adapter_scale, 4) ||
      !aligned(err_flag, 4))
    return MOE_ERR_MISALIGNED;
  const AdapterLinear g{static_cast<const uint16_t*>(x_bf16), static_cast<const uint16_t*>(w_bf16),
                        static_cast<const uint16_t*>(adapter_a_bf16), static_cast<const uint16_t*>(adapter_b_bf16),
                        adapter_ids, adapter_scale, static_cast<uint16_t*>(out_bf16), T, N, K, R, L,
                        act == MOE_ACT_SWIGLU, static_cast<uint8_t*>(workspace), err_flag};
  if (launch_adapter_linear(g, stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

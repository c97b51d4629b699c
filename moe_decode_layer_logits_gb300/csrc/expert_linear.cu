// moe_expert_linear: the products of the routed rows with their experts'
// weights, out[r] = act(W_e x[src(r)]) for the rows r of expert e's segment
// (argument checks; the kernels are in expert_gemm.cuh).
#include "expert_gemm.h"
#include "host_util.h"

namespace moe {

// Checks common to both products.
int check_linear(int64_t N, int64_t K, int32_t act) {
  if (N < 1 || K < 1 || (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU)) return MOE_ERR_INVALID_ARG;
  if (N % (act == MOE_ACT_SWIGLU ? 16 : 8) != 0 || K % 8 != 0 || N > MOE_MAX_DIM || K > MOE_MAX_DIM)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

extern "C" int64_t moe_expert_linear_workspace(int64_t n_rows, int64_t E, int64_t N, int64_t K) {
  if (n_rows < 0 || E < 1 || N < 1 || K < 1) return -1;
  return moe::expert_gemm_workspace(n_rows);
}

extern "C" int moe_expert_linear(const void* x_bf16, int64_t n_x, const int32_t* row_token, const void* w_bf16,
                                 const int32_t* offsets, const int32_t* counts, void* out_bf16, int64_t n_rows,
                                 int64_t E, int64_t N, int64_t K, int32_t act, void* workspace,
                                 int64_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
  using namespace moe;
  if (n_x < 0 || n_rows < 0 || E < 1 || workspace_bytes < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(N, K, act);
  if (st != MOE_OK) return st;
  if (E > MOE_MAX_E || n_x > 0x7FFFFFFFll || n_rows > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  // more tiles than the kernel counts (such an output fits no memory)
  if ((n_rows / 32 + E) * ((N + 63) / 64) > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (!row_token && n_x < n_rows) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if ((n_x > 0 && !x_bf16) || !w_bf16 || !offsets || !counts || !out_bf16) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_expert_linear_workspace(n_rows, E, N, K) || (workspace_bytes > 0 && !workspace))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(out_bf16, 16) || !aligned(workspace, 16) ||
      !aligned(row_token, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(err_flag, 4))
    return MOE_ERR_MISALIGNED;
  const ExpertGemm g{x_bf16, row_token, w_bf16, offsets, counts, out_bf16, n_x, n_rows, E, N, K,
                     act == MOE_ACT_SWIGLU, static_cast<float*>(workspace), err_flag};
  if (launch_expert_gemm(g, stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

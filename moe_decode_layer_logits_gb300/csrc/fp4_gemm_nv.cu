// The 4-bit products: NVFP4, and what both formats share.
#include "fp4_gemm.cuh"

namespace moe {

// (the order of the rows' scales; NVFP4 has more of them than MXFP4)
int64_t fp4_gemm_workspace(int64_t n_rows, int64_t E, int64_t N, int64_t K) {
  return n_rows > 0 && runs_in_pairs(n_rows, E, N, K) ? row_scale_bytes(n_rows, E, K, MOE_FP4_NV) : 0;
}

cudaError_t launch_fp4_gemm_nv(const Fp4Gemm& g, cudaStream_t stream) { return launch_format<MOE_FP4_NV>(g, stream); }

}  // namespace moe

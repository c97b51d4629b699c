// The 4-bit products: MXFP4.
#include "fp4_gemm.cuh"

namespace moe {

cudaError_t launch_fp4_gemm_mx(const Fp4Gemm& g, cudaStream_t stream) { return launch_format<MOE_FP4_MX>(g, stream); }

}  // namespace moe

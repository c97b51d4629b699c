// The calls of the 4-bit operators: argument checks (the kernels are in
// fp4_quant.cu and fp4_gemm.cuh).
#include "expert_gemm.h"
#include "fp4.h"
#include "host_util.h"

namespace moe {

namespace {

int done(cudaError_t e) {
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

// Pieces of 16 elements of one launch, two for each of a block's 128 threads.
constexpr int64_t kMaxPieces = static_cast<int64_t>(0x7FFFFFFF) * 256;

int check_rows(int64_t T, int64_t K, int32_t format) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_fp4(K, format);
  if (st != MOE_OK) return st;
  return T > kMaxPieces / (K / 16) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_products(int64_t N, int64_t K, int32_t format, int32_t act) {
  const int st = check_fp4(K, format);
  return st != MOE_OK ? st : check_linear(N, K, act);
}

}  // namespace
}  // namespace moe

extern "C" int moe_fp4_quantize(const void* x_bf16, const float* global_scale, void* codes, void* scales, int64_t T,
                                int64_t K, int32_t format, cudaStream_t stream) {
  using namespace moe;
  const int st = check_rows(T, K, format);
  if (st != MOE_OK) return st;
  if (global_scale && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(global_scale, 4)) return MOE_ERR_MISALIGNED;
  return done(launch_fp4_quantize(x_bf16, global_scale, codes, scales, T, K, format, stream));
}

extern "C" int moe_fp4_dequantize(const void* codes, const void* scales, const float* global_scale, void* out_bf16,
                                  int64_t T, int64_t K, int32_t format, cudaStream_t stream) {
  using namespace moe;
  const int st = check_rows(T, K, format);
  if (st != MOE_OK) return st;
  if (global_scale && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!codes || !scales || !out_bf16) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(out_bf16, 16) || !aligned(global_scale, 4)) return MOE_ERR_MISALIGNED;
  return done(launch_fp4_dequantize(codes, scales, global_scale, out_bf16, T, K, format, stream));
}

extern "C" int64_t moe_fp4_weight_scales_bytes(int64_t E, int64_t N, int64_t K, int32_t format, int32_t act) {
  using namespace moe;
  if (E < 1 || E > MOE_MAX_E || check_products(N, K, format, act) != MOE_OK) return -1;
  return fp4_weight_scales_bytes(E, N, K, format, act == MOE_ACT_SWIGLU);
}

extern "C" int moe_fp4_weight_scales(const void* scales, void* tiled, int64_t E, int64_t N, int64_t K, int32_t format,
                                     int32_t act, cudaStream_t stream) {
  using namespace moe;
  if (E < 1) return MOE_ERR_INVALID_ARG;
  const int st = check_products(N, K, format, act);
  if (st != MOE_OK) return st;
  if (E > MOE_MAX_E) return MOE_ERR_UNSUPPORTED;
  if (!scales || !tiled) return MOE_ERR_INVALID_ARG;
  if (!aligned(scales, 4) || !aligned(tiled, 16)) return MOE_ERR_MISALIGNED;
  return done(launch_fp4_weight_scales(scales, tiled, E, N, K, format, act == MOE_ACT_SWIGLU, stream));
}

extern "C" int64_t moe_fp4_linear_workspace(int64_t n_rows, int64_t E, int64_t N, int64_t K) {
  if (n_rows < 0 || n_rows > 0x7FFFFFFFll || E < 1 || N < 1 || K < 1 || N > MOE_MAX_DIM || K > MOE_MAX_DIM) return -1;
  return moe::fp4_gemm_workspace(n_rows, E, N, K);
}

namespace moe {
namespace {

// Both products, behind the checks of what only one of them has.
int products(const Fp4Gemm& g, int32_t act, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (g.n_x < 0 || g.n_rows < 0 || g.E < 1 || workspace_bytes < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_products(g.N, g.K, g.format, act);
  if (st != MOE_OK) return st;
  if (g.E > MOE_MAX_E || g.n_x > 0x7FFFFFFFll || g.n_rows > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  // more tiles than the kernel counts (such an output fits no memory)
  if ((g.n_rows / 32 + g.E) * ((g.N + 63) / 64) > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (!g.row_token && g.n_x < g.n_rows) return MOE_ERR_INVALID_ARG;
  if (g.n_rows == 0) return MOE_OK;
  if ((g.n_x > 0 && (!g.x || !g.x_scales)) || !g.w || !g.w_scales || !g.out) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < fp4_gemm_workspace(g.n_rows, g.E, g.N, g.K) || (workspace_bytes > 0 && !workspace)) return MOE_ERR_INVALID_ARG;
  if (!aligned(g.x, 16) || !aligned(g.x_scales, 4) || !aligned(g.w, 16) || !aligned(g.w_scales, 16) || !aligned(g.out, 16) ||
      !aligned(workspace, 16) || !aligned(g.row_token, 4) || !aligned(g.factor, 4) || !aligned(g.offsets, 4) ||
      !aligned(g.counts, 4) || !aligned(g.err_flag, 4))
    return MOE_ERR_MISALIGNED;
  return done(g.format == MOE_FP4_NV ? launch_fp4_gemm_nv(g, stream) : launch_fp4_gemm_mx(g, stream));
}

}  // namespace
}  // namespace moe

extern "C" int moe_fp4_linear(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                              const float* factor, void* out_bf16, int64_t T, int64_t N, int64_t K, int32_t format,
                              int32_t act, void* workspace, int64_t workspace_bytes, int32_t* err_flag,
                              cudaStream_t stream) {
  using namespace moe;
  const Fp4Gemm g{static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales), nullptr,
                  static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales), factor, nullptr, nullptr,
                  out_bf16, T, T, 1, N, K, format, act == MOE_ACT_SWIGLU, workspace, err_flag};
  return products(g, act, workspace, workspace_bytes, stream);
}

extern "C" int moe_fp4_expert_linear(const void* x_codes, const void* x_scales, int64_t n_x, const int32_t* row_token,
                                     const void* w_codes, const void* w_scales, const float* factor,
                                     const int32_t* offsets, const int32_t* counts, void* out_bf16, int64_t n_rows,
                                     int64_t E, int64_t N, int64_t K, int32_t format, int32_t act, void* workspace,
                                     int64_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
  using namespace moe;
  if (n_rows > 0 && (!offsets || !counts)) return MOE_ERR_INVALID_ARG;
  const Fp4Gemm g{static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales), row_token,
                  static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales), factor, offsets, counts,
                  out_bf16, n_x, n_rows, E, N, K, format, act == MOE_ACT_SWIGLU, workspace, err_flag};
  return products(g, act, workspace, workspace_bytes, stream);
}

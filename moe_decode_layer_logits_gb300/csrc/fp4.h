// Microscaled 4-bit floating point: formats, sizes and launches (the kernels
// are in fp4_quant.cu and fp4_gemm.cuh, the calls in fp4_linear.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_tail.h"

namespace moe {

constexpr int kFp4Stage = 256;  // K elements that a stage of the products holds: 128 bytes of codes

// Elements that share a scale.
__host__ __device__ constexpr int fp4_block(int format) { return format == MOE_FP4_NV ? 16 : 32; }

// Scale bytes of a row's stage.
__host__ __device__ constexpr int fp4_stage_scales(int format) { return kFp4Stage / fp4_block(format); }

// MOE_OK if K and format are ones that the operators take.
inline int check_fp4(int64_t K, int32_t format) {
  if (K < 1 || (format != MOE_FP4_NV && format != MOE_FP4_MX)) return MOE_ERR_INVALID_ARG;
  // a row's scales are whole 32-bit words
  if (K % (4 * fp4_block(format)) != 0 || K > MOE_MAX_DIM) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// 128-row tiles of a weight: with SwiGLU 64 outputs each, gate and up rows
// interleaved by 16.
inline int64_t fp4_weight_tiles(int64_t N, bool swiglu) { return swiglu ? (N / 2 + 63) / 64 : (N + 127) / 128; }

inline int64_t fp4_stages(int64_t K) { return (K + kFp4Stage - 1) / kFp4Stage; }

inline int64_t fp4_weight_scales_bytes(int64_t E, int64_t N, int64_t K, int format, bool swiglu) {
  return E * fp4_weight_tiles(N, swiglu) * fp4_stages(K) * 128 * fp4_stage_scales(format);
}

cudaError_t launch_fp4_quantize(const void* x, const float* global_scale, void* codes, void* scales, int64_t T, int64_t K,
                                int format, cudaStream_t stream);
cudaError_t launch_fp4_dequantize(const void* codes, const void* scales, const float* global_scale, void* out, int64_t T,
                                  int64_t K, int format, cudaStream_t stream);
cudaError_t launch_fp4_weight_scales(const void* scales, void* tiled, int64_t E, int64_t N, int64_t K, int format,
                                     bool swiglu, cudaStream_t stream);

struct Fp4Gemm {
  const uint8_t* x;          // [n_x, K / 2]
  const uint8_t* x_scales;   // [n_x, K / block]
  const int32_t* row_token;  // [n_rows] or null
  const uint8_t* w;          // [E, N, K / 2]
  const uint8_t* w_scales;   // as launch_fp4_weight_scales writes them
  const float* factor;       // [E] or null
  const int32_t* offsets;    // [E], or null: one segment of all rows
  const int32_t* counts;     // [E]
  void* out;                 // [n_rows, N or N / 2] BF16
  int64_t n_x, n_rows, E, N, K;
  int format;
  bool swiglu;
  void* workspace;           // of fp4_gemm_workspace() bytes
  int32_t* err_flag;
};

int64_t fp4_gemm_workspace(int64_t n_rows, int64_t E, int64_t N, int64_t K);

cudaError_t launch_fp4_gemm_nv(const Fp4Gemm& g, cudaStream_t stream);
cudaError_t launch_fp4_gemm_mx(const Fp4Gemm& g, cudaStream_t stream);

}  // namespace moe

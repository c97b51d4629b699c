// Products of 4-bit rows with 4-bit weights: the plain kernel.  A block takes
// 32 outputs of an expert; a thread one of them for four of its rows at a time.
#include "common.cuh"
#include "fp4.h"
#include "host_util.h"

namespace moe {

namespace {

__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * static_cast<float>(m) : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
}

template <int FORMAT>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (FORMAT == MOE_FP4_MX)
    return b == 0xFFu ? __uint_as_float(0x7FC00000u) : b > 0 ? __uint_as_float(b << 23) : 0x1p-127f;
  const uint32_t a = b & 0x7Fu;
  const float v = a == 0x7Fu ? __uint_as_float(0x7FC00000u)
                  : a >= 8   ? __uint_as_float(((a >> 3) + 120u) << 23 | (a & 7u) << 20)
                             : static_cast<float>(a) * 0x1p-9f;
  return v;
}

template <int FORMAT>
__global__ void __launch_bounds__(128) fp4_plain_kernel(const Fp4Gemm g, int n_out, int tiles, int stages) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int e = blockIdx.y, o = blockIdx.x * 32 + (threadIdx.x & 31), sub = threadIdx.x >> 5;
  const int64_t beg = g.offsets ? g.offsets[e] : 0, cnt = g.offsets ? g.counts[e] : g.n_rows;
  if (beg < 0 || cnt < 0 || beg + cnt > g.n_rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && g.err_flag) atomicOr(g.err_flag, MOE_FLAG_BAD_INDEX);
    return;
  }
  if (o >= n_out) return;
  const float f = g.factor ? g.factor[e] : 1.f;
  constexpr int B = fp4_block(FORMAT), S = fp4_stage_scales(FORMAT);
  for (int64_t r = beg + sub; r < beg + cnt; r += 4) {
    const int64_t tok = g.row_token ? g.row_token[r] : r;
    float y[2] = {0.f, 0.f};
    if (tok < 0 || tok >= g.n_x) {
      if (g.err_flag) atomicOr(g.err_flag, MOE_FLAG_BAD_INDEX);
    } else {
      for (int part = 0; part < (g.swiglu ? 2 : 1); ++part) {
        const int64_t row = static_cast<int64_t>(e) * g.N + o + part * n_out;
        const int tr = g.swiglu ? (o & 63) / 16 * 32 + part * 16 + (o & 15) : o & 127;
        const uint8_t* ws = g.w_scales + (static_cast<int64_t>(e) * tiles + (g.swiglu ? o / 64 : o / 128)) * stages * 128 * S;
        for (int64_t k = 0; k < g.K; k += B) {
          const int64_t st = k / 256, in = k % 256 / B;
          float sum = 0.f;
          for (int j = 0; j < B; j += 2) {
            const uint32_t a = g.w[(row * g.K + k + j) / 2], b = g.x[(tok * g.K + k + j) / 2];
            sum += code_value(a & 15u) * code_value(b & 15u) + code_value(a >> 4) * code_value(b >> 4);
          }
          y[part] += sum * scale_value<FORMAT>(ws[st * 128 * S + in / 4 * 512 + (tr & 31) * 16 + (tr >> 5) * 4 + (in & 3)]) *
                     scale_value<FORMAT>(g.x_scales[tok * (g.K / B) + k / B]);
        }
        y[part] *= f;
      }
      if (g.swiglu) y[0] = y[0] / (1.f + expf(-y[0])) * y[1];
    }
    static_cast<uint16_t*>(g.out)[r * n_out + o] = static_cast<uint16_t>(pack_bf16x2(y[0], 0.f));
  }
}

}  // namespace

int64_t fp4_gemm_workspace(int64_t) { return 0; }

cudaError_t launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t stream) {
  const int n_out = static_cast<int>(g.swiglu ? g.N / 2 : g.N);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n_out + 31) / 32), static_cast<unsigned>(g.E), 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int tiles = static_cast<int>(fp4_weight_tiles(g.N, g.swiglu)), stages = static_cast<int>(fp4_stages(g.K));
  return g.format == MOE_FP4_NV ? cudaLaunchKernelEx(&cfg, fp4_plain_kernel<MOE_FP4_NV>, g, n_out, tiles, stages)
                                : cudaLaunchKernelEx(&cfg, fp4_plain_kernel<MOE_FP4_MX>, g, n_out, tiles, stages);
}

}  // namespace moe

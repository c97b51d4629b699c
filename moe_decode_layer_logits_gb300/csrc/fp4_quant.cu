// Microscaled 4-bit floating point: BF16 rows to E2M1 codes with a scale for
// each block of neighbours, and back; weights' scales in the products' order.
//
// A thread takes 16 neighbours of a row (an NVFP4 block, half an MXFP4 one), so
// nothing but the MXFP4 maximum crosses threads.  The choices are those of the
// real quotients, not of rounded ones:
//  - the E4M3 scale: a first value from an FP32 product, then the sign of
//    6 m g - amax (m the midpoint to either neighbour) moves it; 6 m has at most 7
//    bits, so one fused multiply-add gives that sign exactly;
//  - the codes: |x| against the seven midpoints times scale times global scale.
//    m s is exact in FP32 (at most 7 bits); times g it is rounded down, and cut to
//    BF16, for the midpoints that go to the lower code, and rounded up for the
//    others, which leaves every comparison with a BF16 number as it was.
// So no quotient is formed, and two elements are compared at once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp4.h"
#include "host_util.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr uint8_t kNanE4m3 = 0x7F, kNanE8m0 = 0xFF;

__device__ __forceinline__ float e4m3_value(int byte) {  // of a byte without sign
  return byte >= 8 ? __uint_as_float(static_cast<uint32_t>((byte >> 3) + 120) << 23 | static_cast<uint32_t>(byte & 7) << 20)
                   : static_cast<float>(byte) * 0x1p-9f;
}

__device__ __forceinline__ float e8m0_value(int byte) {
  return byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
}

// Global scales outside this range make NaN: inside it no product above ends in a
// subnormal number or overflows.
__device__ __forceinline__ bool usable(float g) { return g >= 0x1p-100f && g <= 0x1p100f; }

// e4m3(amax / (6 g)), nearest even, at most 448.
__device__ __forceinline__ int e4m3_scale(float amax, float g) {
  const int c = __nv_cvt_float_to_fp8(amax / (6.f * g), __NV_SATFINITE, __NV_E4M3);
  if (c < 126) {
    const float above = fmaf((e4m3_value(c) + e4m3_value(c + 1)) * 3.f, g, -amax);
    if (above < 0.f || (above == 0.f && (c & 1))) return c + 1;
  }
  if (c > 0) {
    const float below = fmaf((e4m3_value(c - 1) + e4m3_value(c)) * 3.f, g, -amax);
    if (below > 0.f || (below == 0.f && (c & 1))) return c - 1;
  }
  return c;
}

// The same BF16 number twice: x > it if and only if x > m s g (EVEN_BELOW: a tie
// goes to the lower code), or x >= m s g.
template <bool EVEN_BELOW>
__device__ __forceinline__ uint32_t threshold(float ms, float g) {
  uint32_t b;
  if (EVEN_BELOW) b = __float_as_uint(__fmul_rd(ms, g)) >> 16;
  else b = ((__float_as_uint(__fmul_ru(ms, g)) + 0xFFFFu) >> 16) - 1;
  return b | b << 16;
}

__device__ __forceinline__ uint32_t greater2(uint32_t a, uint32_t b) {  // 0xFFFF in each half where a > b
  return __hgt2_mask(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
}

__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t yes, uint32_t no) { return (yes & mask) | (no & ~mask); }

template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
fp4_quantize_kernel(const uint4* x, const float* global_scale, uint2* codes, uint8_t* scales, int64_t pieces) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const bool live = i < pieces;  // (a block's pieces lie in one warp)
  const float g = FORMAT == MOE_FP4_NV && global_scale ? __ldg(global_scale) : 1.f;
  uint4 v[2] = {};
  if (live) {
    v[0] = ld_stream16(x + 2 * i);
    v[1] = ld_stream16(x + 2 * i + 1);
  }
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);  // the largest |x|, as BF16 bits
  if (FORMAT == MOE_FP4_MX) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  bool finite = top < 0x7F80u;
  int scale;
  float s;
  if (FORMAT == MOE_FP4_NV) {
    finite = finite && usable(g);
    scale = finite ? e4m3_scale(__uint_as_float(top << 16), g) : kNanE4m3;
    s = e4m3_value(scale);
  } else {
    scale = finite ? max(static_cast<int>(top >> 7) - 2, 0) : kNanE8m0;  // floor(log2) - 2, biased
    s = e8m0_value(scale);
  }
  if (!live) return;
  uint32_t out[2] = {0u, 0u};
  if (finite && (FORMAT == MOE_FP4_MX || scale > 0)) {
    const uint32_t t0 = threshold<true>(0.25f * s, g), t1 = threshold<false>(0.75f * s, g),
                   t2 = threshold<true>(1.25f * s, g), t3 = threshold<false>(1.75f * s, g),
                   t4 = threshold<true>(2.5f * s, g), t5 = threshold<false>(3.5f * s, g),
                   t6 = threshold<true>(5.f * s, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = w[j] & 0x7FFF7FFFu;
      const uint32_t b2 = greater2(a, t3);
      const uint32_t b1 = greater2(a, pick(b2, t5, t1));
      const uint32_t b0 = greater2(a, pick(b1, pick(b2, t6, t2), pick(b2, t4, t0)));
      const uint32_t c = (b2 & 0x00040004u) | (b1 & 0x00020002u) | (b0 & 0x00010001u) | (w[j] >> 12 & 0x00080008u);
      out[j >> 2] |= ((c | c >> 12) & 0xFFu) << (8 * (j & 3));
    }
  }
  codes[i] = make_uint2(out[0], out[1]);
  if (FORMAT == MOE_FP4_NV) scales[i] = static_cast<uint8_t>(scale);
  else if ((i & 1) == 0) scales[i >> 1] = static_cast<uint8_t>(scale);
}

// v g, as an FP32 number that rounds to BF16 like the exact product: cut, with
// the last bit set where something was cut off.
__device__ __forceinline__ float product_to_odd(float v, float g) {
  const float p = __fmul_rz(v, g);
  return fmaf(v, g, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
fp4_dequantize_kernel(const uint2* codes, const uint8_t* scales, const float* global_scale, uint4* out, int64_t pieces) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const float g = FORMAT == MOE_FP4_NV && global_scale ? __ldg(global_scale) : 1.f;
  const uint2 c = codes[i];
  const int byte = scales[FORMAT == MOE_FP4_NV ? i : i >> 1];
  float s;
  if (FORMAT == MOE_FP4_NV) s = (byte & 0x7F) == kNanE4m3 ? __uint_as_float(0x7FC00000u) : e4m3_value(byte & 0x7F);
  else s = byte == kNanE8m0 ? __uint_as_float(0x7FC00000u) : e8m0_value(byte);
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t two = ((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xFFu;
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = two >> (4 * h), m = k & 7u;
      // 0, 0.5, then 1 bit of mantissa
      const float v = m < 2 ? 0.5f * static_cast<float>(m)
                            : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
      f[h] = (k & 8u ? -v : v) * s;
      if (FORMAT == MOE_FP4_NV) f[h] = product_to_odd(f[h], g);
    }
    o[j] = pack_bf16x2(f[0], f[1]);
  }
  out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
  out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Scales [E, N, K / block] to one piece of 128 rows x a stage after the other:
// [expert][weight tile][stage][word][row % 32][row / 32], words of four
// neighbouring scales, zeros outside N and K.  That is what a copy into the
// tensor memory wants, and one bulk copy brings a stage's piece.
template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
fp4_weight_scales_kernel(const uint32_t* scales, uint32_t* tiled, int64_t words, int tiles, int stages, int N, int K,
                         int swiglu) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int kWords = fp4_stage_scales(FORMAT) / 4, kElements = 4 * fp4_block(FORMAT);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= words) return;
  const int j = static_cast<int>(i & 3), lane = static_cast<int>(i >> 2 & 31);
  const int64_t piece = i >> 7;
  const int word = static_cast<int>(piece % kWords);
  const int64_t q = piece / kWords;
  const int stage = static_cast<int>(q % stages);
  const int64_t m = q / stages % tiles, e = q / stages / tiles;
  int64_t row;
  bool live;
  if (swiglu) {
    const int64_t o = m * 64 + j * 16 + (lane & 15);
    live = o < N / 2;
    row = o + (lane >= 16 ? N / 2 : 0);
  } else {
    row = m * 128 + j * 32 + lane;
    live = row < N;
  }
  const int col = stage * kWords + word, cols = K / kElements;
  tiled[i] = live && col < cols ? scales[(e * N + row) * cols + col] : 0u;
}

template <typename F, typename... A>
cudaError_t launch_threads(F* kernel, int64_t n, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_fp4_quantize(const void* x, const float* global_scale, void* codes, void* scales, int64_t T, int64_t K,
                                int format, cudaStream_t stream) {
  const int64_t pieces = T * (K / 16);
  const auto xs = static_cast<const uint4*>(x);
  const auto c = static_cast<uint2*>(codes);
  const auto s = static_cast<uint8_t*>(scales);
  return format == MOE_FP4_NV ? launch_threads(fp4_quantize_kernel<MOE_FP4_NV>, pieces, stream, xs, global_scale, c, s, pieces)
                              : launch_threads(fp4_quantize_kernel<MOE_FP4_MX>, pieces, stream, xs, global_scale, c, s, pieces);
}

cudaError_t launch_fp4_dequantize(const void* codes, const void* scales, const float* global_scale, void* out, int64_t T,
                                  int64_t K, int format, cudaStream_t stream) {
  const int64_t pieces = T * (K / 16);
  const auto c = static_cast<const uint2*>(codes);
  const auto s = static_cast<const uint8_t*>(scales);
  const auto o = static_cast<uint4*>(out);
  return format == MOE_FP4_NV ? launch_threads(fp4_dequantize_kernel<MOE_FP4_NV>, pieces, stream, c, s, global_scale, o, pieces)
                              : launch_threads(fp4_dequantize_kernel<MOE_FP4_MX>, pieces, stream, c, s, global_scale, o, pieces);
}

cudaError_t launch_fp4_weight_scales(const void* scales, void* tiled, int64_t E, int64_t N, int64_t K, int format,
                                     bool swiglu, cudaStream_t stream) {
  const int64_t words = fp4_weight_scales_bytes(E, N, K, format, swiglu) / 4;
  const int tiles = static_cast<int>(fp4_weight_tiles(N, swiglu)), stages = static_cast<int>(fp4_stages(K));
  const auto s = static_cast<const uint32_t*>(scales);
  const auto t = static_cast<uint32_t*>(tiled);
  return format == MOE_FP4_NV
             ? launch_threads(fp4_weight_scales_kernel<MOE_FP4_NV>, words, stream, s, t, words, tiles, stages,
                              static_cast<int>(N), static_cast<int>(K), swiglu ? 1 : 0)
             : launch_threads(fp4_weight_scales_kernel<MOE_FP4_MX>, words, stream, s, t, words, tiles, stages,
                              static_cast<int>(N), static_cast<int>(K), swiglu ? 1 : 0);
}

}  // namespace moe

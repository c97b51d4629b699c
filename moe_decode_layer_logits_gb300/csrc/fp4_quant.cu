// Microscaled 4-bit floating point: BF16 rows to E2M1 codes with a scale for
// each block of neighbours, and back; weights' scales in the products' order.
//
// A thread takes pieces of 16 neighbours of a row (an NVFP4 block, half an MXFP4
// one), so nothing but the MXFP4 maximum crosses threads.  The choices are those
// of the real quotients, not of rounded ones:
//  - the E4M3 scale: a first value from an FP32 product, then the sign of
//    6 m g - amax, m the midpoint to the neighbour on the product's side, keeps or
//    moves it; 6 m has at most 7 bits, so one fused multiply-add has that sign
//    exactly;
//  - the codes, by the conversion instruction from an FP32 quotient: where a midpoint
//    times scale times global scale lies beside every BF16 number, the quotient's few
//    roundings leave it on the right side.  Where one lies next to a BF16 number, or
//    on it, the quotient is moved by 2^-20 to the side on which the real one is (or
//    on which a tie ends).  Both depend on mantissas alone, 4 of midpoints times 8 of
//    scales, so a warp asks once.  (MXFP4's quotients are exact.)
//  - where the midpoints of a block's scale want both sides, as without a global
//    scale, |x| is compared with the seven midpoints times scale times global scale.
//    m s is exact in FP32 (at most 7 bits); times g it is rounded down, and cut to
//    BF16, for the midpoints that go to the lower code, and rounded up for the
//    others, which leaves every comparison with a BF16 number as it was.  Two
//    elements are compared at once.  The values of
// the eight codes of a block, rounded to BF16 once, are a table of 16 bytes on the
// way back, from which byte permutations pick four at a time.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp4.h"
#include "host_util.h"

namespace moe {

namespace {

constexpr int kThreads = 128;
constexpr int kPieces = 2;  // of a thread, loaded at once
constexpr uint8_t kNanE4m3 = 0x7F, kNanE8m0 = 0xFF;

__device__ __forceinline__ float e4m3_value(int byte) {  // of a byte without sign
  return byte >= 8 ? __uint_as_float(static_cast<uint32_t>((byte >> 3) + 120) << 23 | static_cast<uint32_t>(byte & 7) << 20)
                   : static_cast<float>(byte) * 0x1p-9f;
}

__device__ __forceinline__ float e8m0_value(int byte) {
  return byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
}

// Global scales outside this range make NaN: inside it no product here ends in a
// subnormal number or overflows.
__device__ __forceinline__ bool usable(float g) { return g >= 0x1p-100f && g <= 0x1p100f; }

// e4m3(amax / (6 g)), nearest even, at most 448; about = 1 / (6 g) within a few
// roundings.
__device__ __forceinline__ int e4m3_scale(float amax, float g, float about) {
  const float q = amax * about;
  const int c = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  // far from a midpoint (by 16 units of FP32's last place), as nearly always
  if (c > 8 && ((__float_as_uint(q) + 0x80010u) & 0xFFFE0u) != 0u) return c;
  const float v = e4m3_value(c);
  const bool up = q >= v;
  if (up && c == 126) return c;
  if (!up && c == 0) return c;
  // Half a step up or down: half of the lowest mantissa bit in FP32's bits, across
  // the powers of two as well; below 2^-6 the steps are 2^-9.
  const float m = c > 8 || (up && c == 8) ? __int_as_float(__float_as_int(v) + (up ? 1 << 19 : -(1 << 19))) : v + (up ? 0x1p-10f : -0x1p-10f);
  const float d = fmaf(6.f * m, g, -amax);  // > 0: amax lies below the midpoint
  const bool tie = d == 0.f && (c & 1);
  return up ? c + (d < 0.f || tie ? 1 : 0) : c - (d > 0.f || tie ? 1 : 0);
}

// The same BF16 number twice: x > it if and only if x > m s g (EVEN_BELOW: a tie
// goes to the lower code), or x >= m s g.
template <bool EVEN_BELOW>
__device__ __forceinline__ uint32_t threshold(float ms, float g) {
  if (EVEN_BELOW) return __byte_perm(__float_as_uint(__fmul_rd(ms, g)), 0, 0x3232);
  return __byte_perm(__float_as_uint(__fmul_ru(ms, g)) - 1u, 0, 0x3232);
}

__device__ __forceinline__ uint32_t greater2(uint32_t a, uint32_t b) {  // 0xFFFF in each half where a > b
  return __hgt2_mask(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
}

__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t yes, uint32_t no) { return (yes & mask) | (no & ~mask); }

// 4 [b2] + 2 [b1] + [b0] in each half, from masks of 0xFFFF.  As numbers the masks
// with bits h and l are 2^16 (l - h) - l, so their weighted sum times -(2^16 + 1)
// is 2^16 of the high code plus the low one.  (Multiply-adds, as the logic pipe
// bounds this way: T = 8192 33.3 -> 30.4 us.)
__device__ __forceinline__ uint32_t bits_of(uint32_t b2, uint32_t b1, uint32_t b0) {
  uint32_t s;
  asm("mad.lo.u32 %0, %1, 2, %2;" : "=r"(s) : "r"(b1), "r"(b0));
  asm("mad.lo.u32 %0, %1, 4, %2;" : "=r"(s) : "r"(b2), "r"(s));
  return s * 0xFFFEFFFFu;
}

// Which of the 32 pairs of mantissas, of m (1, 1.25, 1.5, 1.75: bits 0, 1) and s (1 to
// 1.875: bits 2 to 4), have an m s g within 32 units of FP32's last place of a BF16
// number, where an FP32 quotient x / (s g) (whose roundings are some 2^-22, 2 to 4
// units) may lie on the other side of m than the real one: `up` if the real one is
// above it, or on it and the code above is even, `down` otherwise.
struct Sides {
  uint32_t up, down;
};
__device__ __forceinline__ Sides sides_of(float g) {
  const int lane = threadIdx.x & 31;
  const float ms = (1.f + 0.25f * static_cast<float>(lane & 3)) * (1.f + 0.125f * static_cast<float>(lane >> 2));
  const uint32_t bits = __float_as_uint(ms * g), low = bits & 0xFFFFu;
  const bool near = low <= 32u || low >= 0x10000u - 32u;
  const float d = fmaf(ms, g, -__uint_as_float((bits + 0x8000u) & 0xFFFF0000u));  // m s g less that number
  const bool above = d < 0.f || (d == 0.f && (lane & 3) >= 2);
  return {__ballot_sync(0xFFFFFFFFu, near && above), __ballot_sync(0xFFFFFFFFu, near && !above)};
}

// One piece: 16 BF16 numbers to 8 bytes of codes; `scale` of its block.
template <int FORMAT>
__device__ __forceinline__ uint2 quantize_piece(const uint4 (&v)[2], float g, float about, bool usable_g, Sides sides, int& scale) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);  // the largest |x|, as BF16 bits
  if (FORMAT == MOE_FP4_MX) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  float s;
  bool codes;  // (a block that is not finite has none, nor one whose scale is zero)
  if (FORMAT == MOE_FP4_NV) {
    const bool finite = top < 0x7F80u && usable_g;
    scale = finite ? e4m3_scale(__uint_as_float(top << 16), g, about) : kNanE4m3;
    codes = finite && scale > 0;
    s = e4m3_value(scale);
  } else {
    codes = top < 0x7F80u;
    scale = codes ? max(static_cast<int>(top >> 7) - 2, 0) : kNanE8m0;  // floor(log2) - 2, biased
    s = e8m0_value(scale);
  }
  if (!codes) return make_uint2(0u, 0u);
  // the mantissa's three bits (of a scale below 2^-6: those behind its first one)
  const int at = 4 * (scale >= 8 ? scale & 7 : static_cast<int>(0x64204000u >> (4 * scale) & 7u));
  const bool up = FORMAT == MOE_FP4_NV && (sides.up >> at & 15u) != 0u, down = FORMAT == MOE_FP4_NV && (sides.down >> at & 15u) != 0u;
  if (!(up && down)) {
    float inverse;
    if (FORMAT == MOE_FP4_MX) inverse = __uint_as_float(static_cast<uint32_t>(254 - scale) << 23);
    else inverse = __frcp_rn(s * g) * (up ? 1.f + 0x1p-20f : down ? 1.f - 0x1p-20f : 1.f);
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 q = make_float2(bf16lo(w[j]) * inverse, bf16hi(w[j]) * inverse);
      out[j >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(q, __NV_E2M1, cudaRoundNearest)) << (8 * (j & 3));
    }
    return make_uint2(out[0], out[1]);
  }
  const uint32_t t0 = threshold<true>(0.25f * s, g), t1 = threshold<false>(0.75f * s, g), t2 = threshold<true>(1.25f * s, g),
                 t3 = threshold<false>(1.75f * s, g), t4 = threshold<true>(2.5f * s, g), t5 = threshold<false>(3.5f * s, g),
                 t6 = threshold<true>(5.f * s, g);
  uint32_t c[8];  // each: code of the even element, and of the odd one 16 bits above
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = w[j] & 0x7FFF7FFFu;
    const uint32_t b2 = greater2(a, t3);
    const uint32_t b1 = greater2(a, pick(b2, t5, t1));
    const uint32_t b0 = greater2(a, pick(b1, pick(b2, t6, t2), pick(b2, t4, t0)));
    c[j] = (w[j] >> 12 & 0x00080008u) | bits_of(b2, b1, b0);
  }
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t* k = c + 4 * h;
    const uint32_t even = __byte_perm(k[0], k[2], 0x5410) + (__byte_perm(k[1], k[3], 0x5410) << 8);
    const uint32_t odd = __byte_perm(k[0], k[2], 0x7632) + (__byte_perm(k[1], k[3], 0x7632) << 8);
    out[h] = even + (odd << 4);
  }
  return make_uint2(out[0], out[1]);
}

// Measured, T = 8192, K = 6144 (129 MB): NVFP4 21.7 us (5.9 TB/s, 89% of the copy
// rate), MXFP4 20.7, HBM; by comparisons, as without a global scale, 30.6 (the logic
// pipe).
template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
fp4_quantize_kernel(const uint4* x, const float* global_scale, uint2* codes, uint8_t* scales, int64_t pieces) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;  // (a block's pieces lie in one warp)
  uint4 v[kPieces][2] = {};
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t i = first + k * kThreads;
    if (i < pieces) {
      v[k][0] = ld_stream16(x + 2 * i);
      v[k][1] = ld_stream16(x + 2 * i + 1);
    }
  }
  const float g = FORMAT == MOE_FP4_NV && global_scale ? __ldg(global_scale) : 1.f;
  const bool usable_g = usable(g);
  const float about = 1.f / (6.f * g);
  const Sides sides = FORMAT == MOE_FP4_NV ? sides_of(g) : Sides{0u, 0u};
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t i = first + k * kThreads;
    int scale;
    const uint2 c = quantize_piece<FORMAT>(v[k], g, about, usable_g, sides, scale);
    if (i < pieces) {  // (no thread leaves before the others' shuffles)
      codes[i] = c;
      if (FORMAT == MOE_FP4_NV) scales[i] = static_cast<uint8_t>(scale);
      else if ((i & 1) == 0) scales[i >> 1] = static_cast<uint8_t>(scale);
    }
  }
}

// v g, as an FP32 number that rounds to BF16 like the exact product: cut, with
// the last bit set where something was cut off.
__device__ __forceinline__ float product_to_odd(float v, float g) {
  const float p = __fmul_rz(v, g);
  return fmaf(v, g, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// Measured, T = 8192, K = 6144: 21.8 us (129 MB: 5.9 TB/s, 88% of the copy rate).
template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
fp4_dequantize_kernel(const uint2* codes, const uint8_t* scales, const float* global_scale, uint4* out, int64_t pieces) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  uint2 c[kPieces] = {};
  int byte[kPieces] = {};
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t i = first + k * kThreads;
    if (i < pieces) {
      c[k] = codes[i];
      byte[k] = scales[FORMAT == MOE_FP4_NV ? i : i >> 1];
    }
  }
  const float g = FORMAT == MOE_FP4_NV && global_scale ? __ldg(global_scale) : 1.f;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t i = first + k * kThreads;
    if (i >= pieces) break;
    float s;
    if (FORMAT == MOE_FP4_NV) s = (byte[k] & 0x7F) == kNanE4m3 ? __uint_as_float(0x7FC00000u) : e4m3_value(byte[k] & 0x7F);
    else s = byte[k] == kNanE8m0 ? __uint_as_float(0x7FC00000u) : e8m0_value(byte[k]);
    // the values of codes 0 .. 7
    const float m[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = FORMAT == MOE_FP4_NV ? product_to_odd(m[j] * s, g) : m[j] * s;
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    const uint32_t low0 = __byte_perm(t[0], t[1], 0x6420), low1 = __byte_perm(t[2], t[3], 0x6420),
                   high0 = __byte_perm(t[0], t[1], 0x7531), high1 = __byte_perm(t[2], t[3], 0x7531);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // four elements
      const uint32_t four = (j < 2 ? c[k].x : c[k].y) >> (16 * (j & 1)), at = four & 0x7777u;
      const uint32_t spread = __byte_perm(four, 0, 0x1100);  // each byte twice
      const uint32_t sign = (spread << 4 & 0x00800080u) | (spread & 0x80008000u);
      const uint32_t low = __byte_perm(low0, low1, at), high = __byte_perm(high0, high1, at) | sign;
      o[2 * j] = __byte_perm(low, high, 0x5140);
      o[2 * j + 1] = __byte_perm(low, high, 0x7362);
    }
    out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
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
cudaError_t launch_threads(F* kernel, int64_t n, int per, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n + kThreads * per - 1) / (kThreads * per)), 1, 1);
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
  return format == MOE_FP4_NV ? launch_threads(fp4_quantize_kernel<MOE_FP4_NV>, pieces, kPieces, stream, xs, global_scale, c, s, pieces)
                              : launch_threads(fp4_quantize_kernel<MOE_FP4_MX>, pieces, kPieces, stream, xs, global_scale, c, s, pieces);
}

cudaError_t launch_fp4_dequantize(const void* codes, const void* scales, const float* global_scale, void* out, int64_t T,
                                  int64_t K, int format, cudaStream_t stream) {
  const int64_t pieces = T * (K / 16);
  const auto c = static_cast<const uint2*>(codes);
  const auto s = static_cast<const uint8_t*>(scales);
  const auto o = static_cast<uint4*>(out);
  return format == MOE_FP4_NV ? launch_threads(fp4_dequantize_kernel<MOE_FP4_NV>, pieces, kPieces, stream, c, s, global_scale, o, pieces)
                              : launch_threads(fp4_dequantize_kernel<MOE_FP4_MX>, pieces, kPieces, stream, c, s, global_scale, o, pieces);
}

cudaError_t launch_fp4_weight_scales(const void* scales, void* tiled, int64_t E, int64_t N, int64_t K, int format,
                                     bool swiglu, cudaStream_t stream) {
  const int64_t words = fp4_weight_scales_bytes(E, N, K, format, swiglu) / 4;
  const int tiles = static_cast<int>(fp4_weight_tiles(N, swiglu)), stages = static_cast<int>(fp4_stages(K));
  const auto s = static_cast<const uint32_t*>(scales);
  const auto t = static_cast<uint32_t*>(tiled);
  return format == MOE_FP4_NV
             ? launch_threads(fp4_weight_scales_kernel<MOE_FP4_NV>, words, 1, stream, s, t, words, tiles, stages,
                              static_cast<int>(N), static_cast<int>(K), swiglu ? 1 : 0)
             : launch_threads(fp4_weight_scales_kernel<MOE_FP4_MX>, words, 1, stream, s, t, words, tiles, stages,
                              static_cast<int>(N), static_cast<int>(K), swiglu ? 1 : 0);
}

}  // namespace moe

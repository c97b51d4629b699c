// moe_group_topk_route: top-k routing by scores, one warp per token.
//
//   s = sigmoid(l)  or  softmax(l) over all E experts
//   c = s + bias    (without a bias the order of the choice is that of l)
//   group score = sum of the group's group_top largest c (or s without a bias)
//   ids = the k largest c inside the topk_group best groups
//   w   = routed_scale * s[ids] (/ their sum)
//
// Equal values go to the lower group and the lower expert.  The choice is
// made in 64 bits: with a bias the gaps between neighbours of a row come close
// to 2^-24 in every few thousand rows.
#include "host_util.h"
#include "common.cuh"

namespace moe {

struct GroupRouteParams {
  const float* logits;
  const float* bias;  // [E] or null
  int32_t* ids;
  float* w;
  int T, E, k;
  int n_group, topk_group, group_top;
  int softmax, renorm;
  float scale;
};

constexpr int kGroupRouteWarps = 4;  // tokens per CTA

__device__ __forceinline__ double warp_max_f64(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmax(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// The choice of one token in 64 bits.  `c` and `taken` are this warp's shared
// memory: E values and E flags.  Lane j < k gets the j-th id and its score.
__device__ __noinline__ void group_select_f64(const GroupRouteParams& p, const float* __restrict__ row, double* sc,
                                              double* key, int& id, double& score) {
  const int lane = threadIdx.x & 31;
  const double inf = __longlong_as_double(0x7FF0000000000000ll);
  // scores
  double m = -inf;
  for (int i = lane; i < p.E; i += 32) {
    const float l = row[i];
    const double z = isnan(l) ? -inf : static_cast<double>(l);
    key[i] = z;
    m = fmax(m, z);
  }
  double sum = 1.0;
  if (p.softmax) {
    m = warp_max_f64(m);
    double part = 0.0;
    for (int i = lane; i < p.E; i += 32) {
      const double z = key[i];
      const double e = m == -inf ? 0.0 : z == m ? 1.0 : exp(z - m);
      sc[i] = e;
      part += e;
    }
    sum = warp_sum_f64(part);
    if (sum == 0.0) sum = 1.0;
  }
  for (int i = lane; i < p.E; i += 32) {
    const double s = p.softmax ? sc[i] / sum : 1.0 / (1.0 + exp(-key[i]));
    sc[i] = s;
    if (p.bias) {
      const double c = s + static_cast<double>(p.bias[i]);
      key[i] = isnan(c) ? -inf : c;
    }
  }
  __syncwarp();
  // groups: the worst ones are taken out (their keys become NaN)
  const int size = p.E / p.n_group;
  if (p.topk_group < p.n_group) {
    double gs = -inf;
    if (lane < p.n_group) {
      const bool by_key = p.bias != nullptr || p.group_top == 1;
      double b1 = -inf, b2 = -inf;
      for (int i = lane * size; i < (lane + 1) * size; ++i) {
        const double v = by_key ? key[i] : sc[i];
        if (v > b1) { b2 = b1; b1 = v; }
        else if (v > b2) b2 = v;
      }
      gs = p.group_top == 2 && size > 1 ? b1 + b2 : b1;
      if (isnan(gs)) gs = -inf;
    }
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const double o = __shfl_sync(0xFFFFFFFFu, gs, g);
      rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
    }
    const unsigned in = __ballot_sync(0xFFFFFFFFu, lane < p.n_group && rank < p.topk_group);
    for (int i = lane; i < p.E; i += 32)
      if (!((in >> (i / size)) & 1u)) key[i] = __longlong_as_double(0x7FF8000000000000ll);
    __syncwarp();
  }
  // k rounds: the largest key, the lowest expert among equals
  id = 0;
  score = 0.0;
  for (int r = 0; r < p.k; ++r) {
    double b = -inf;
    int at = 0x7FFFFFFF;
    for (int i = lane; i < p.E; i += 32) {
      const double v = key[i];
      if (v > b || (v == b && i < at)) { b = v; at = i; }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ob = __shfl_xor_sync(0xFFFFFFFFu, b, off);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, off);
      if (oa != 0x7FFFFFFF && (at == 0x7FFFFFFF || ob > b || (ob == b && oa < at))) { b = ob; at = oa; }
    }
    if (lane == r) { id = at; score = sc[at]; }
    __syncwarp();
    if (lane == 0) key[at] = __longlong_as_double(0x7FF8000000000000ll);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kGroupRouteWarps * 32) group_route_kernel(const GroupRouteParams p) {
  extern __shared__ __align__(16) double group_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGroupRouteWarps + warp;
  allow_dependent_launch();
  grid_dependency_wait();
  if (t >= p.T) return;
  double* sc = group_smem + static_cast<size_t>(warp) * 2 * p.E;
  int id;
  double s;
  group_select_f64(p, p.logits + t * p.E, sc, sc + p.E, id, s);
  double w = lane < p.k ? s : 0.0;
  if (p.renorm) {
    const double sum = warp_sum_f64(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = id;
    p.w[t * p.k + lane] = static_cast<float>(static_cast<double>(p.scale) * w);
  }
}

}  // namespace moe

extern "C" int moe_group_topk_route(const float* logits, const float* bias, int32_t* topk_ids, float* topk_w,
                                    int64_t T, int64_t E, int32_t k, int32_t n_group, int32_t topk_group,
                                    int32_t group_top, int32_t score_fn, int32_t renormalize, float routed_scale,
                                    cudaStream_t stream) {
  using namespace moe;
  if (T < 0 || E < 1 || k < 1 || k > MOE_MAX_K || n_group < 1 || topk_group < 1 || topk_group > n_group ||
      E % n_group != 0 || (group_top != 1 && group_top != 2) ||
      (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) || (renormalize != 0 && renormalize != 1) ||
      !isfinite(routed_scale) || k > E / n_group * topk_group)
    return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || n_group > MOE_MAX_GROUPS || T > (static_cast<int64_t>(1) << 30)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return MOE_ERR_MISALIGNED;
  GroupRouteParams p{logits, bias, topk_ids, topk_w, static_cast<int>(T), static_cast<int>(E), k, n_group,
                     topk_group, group_top, score_fn == MOE_SCORE_SOFTMAX, renormalize, routed_scale};
  const size_t smem = static_cast<size_t>(kGroupRouteWarps) * 2 * p.E * sizeof(double);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(group_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
          cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((T + kGroupRouteWarps - 1) / kGroupRouteWarps), 1, 1);
  cfg.blockDim = dim3(kGroupRouteWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, group_route_kernel, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

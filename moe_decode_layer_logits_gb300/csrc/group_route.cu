// moe_group_topk_route: top-k routing by scores, one warp per token.
//
//   s = sigmoid(l)  or  softmax(l) over all E experts
//   c = s + bias    (without a bias the order of the choice is that of l)
//   group score = sum of the group's group_top largest c (or s without a bias)
//   ids = the k largest c inside the topk_group best groups
//   w   = routed_scale * s[ids] (/ their sum)
//
// Equal values go to the lower group and the lower expert.
//
// The choice is that of the formula in 64 bits, made in 32 wherever 32 can
// make it: the FP32 choice values carry a known error, and where two
// neighbours of the order that decides the result lie closer than it, the
// token's candidates (or, for groups and softmax with a bias, the whole row)
// are compared again in 64 bits.  With sigmoid scores of Gaussian logits and a
// bias that is one row in some thousands; in 64 bits throughout, T = 8192 took
// 280 us.  Without a bias the order is that of the logits and is exact.
//
// One token is a chain of dependent warp steps (scores, group scores, group
// choice, a lower bound for the k-th value, ranks among the values above it),
// so small batches are bound by its latency and large ones by its
// instructions; the data is 4 E bytes a token.
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
constexpr int kCandidates = 192;     // longest candidate list; a longer one (ties) goes to 64 bits

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

// The choice of one token in 64 bits.  `sc` and `key` are E values each of this
// warp's shared memory.  Lane j < k gets the j-th id and its score.
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

// Order-preserving key of a float without NaN; -0 and +0 share one.
__device__ __forceinline__ uint32_t order_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u << 1) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Adds v to the two largest values b1 >= b2 so far.
__device__ __forceinline__ void top_two(float& b1, float& b2, float v) {
  b2 = fmaxf(b2, fminf(b1, v));
  b1 = fmaxf(b1, v);
}

// The two halves of a candidate: a larger value is the better choice (larger
// key, then lower expert).
__device__ __forceinline__ uint64_t candidate(float v, int expert) {
  return (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(0xFFFFFFFFu - static_cast<uint32_t>(expert));
}
__device__ __forceinline__ int candidate_expert(uint64_t c) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(c)); }

// Shared memory of one warp, in bytes: the larger of the 32-bit selection's
// arrays and the 64-bit one's.
__host__ __device__ constexpr int route_list_at(int E) { return (E * 4 + (E + E / 32 + 1) * 4 + 15) / 16 * 16; }
__host__ __device__ constexpr int route_smem(int E) {
  const int fast = route_list_at(E) + (kCandidates + 40) * 8 + 128, slow = E * 16;
  return (fast > slow ? fast : slow) / 16 * 16 + 16;
}

template <int EPL>
__global__ void __launch_bounds__(kGroupRouteWarps * 32) group_route_kernel(const GroupRouteParams p) {
  extern __shared__ __align__(16) uint8_t route_mem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGroupRouteWarps + warp;
  const float inf = __int_as_float(0x7F800000);
  allow_dependent_launch();
  // the bias is a parameter, but it too is read after the wait: a balancing
  // step may just have written it
  grid_dependency_wait();
  if (t >= p.T) return;
  uint8_t* mem = route_mem + static_cast<size_t>(warp) * route_smem(p.E);
  float* sv = reinterpret_cast<float*>(mem);         // [E] scores
  float* kv = sv + p.E;                              // [E + E / 32] choice values, one word of padding per 32
  uint64_t* list = reinterpret_cast<uint64_t*>(mem + route_list_at(p.E));
  uint64_t* best = list + kCandidates;               // [k + 1]
  int* chosen = reinterpret_cast<int*>(best + 40);   // [32] groups that stay
  const float* row = p.logits + t * p.E;

  // scores and choice values; `doubt`: how far apart two choice values of
  // this row must lie, beside 2^-22 of their size, to be in the right order
  float key[EPL];
  int num[EPL];  // the expert of each key; -1: none
  float m = -inf;
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    const int i = lane + 32 * s;
    num[s] = i < p.E ? i : -1;
    key[s] = i < p.E ? row[i] : -inf;
    if (isnan(key[s])) key[s] = -inf;
    m = fmaxf(m, key[s]);
  }
  float inv = 1.f;
  if (p.softmax) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    float z = 0.f;
#pragma unroll
    for (int s = 0; s < EPL; ++s)
      if (num[s] >= 0 && m > -inf) z += key[s] == m ? 1.f : expf(key[s] - m);
    z = warp_sum(z);
    inv = z > 0.f ? 1.f / z : 0.f;
  }
  // Sigmoid: expf 2 ulp, sum, quotient: within 2^-22 of a value below 1.  A
  // softmax term: 2^-24 (|l - m| + E / 32 + 12) of itself, and s |l - m| < 1.
  // Two values: twice that.
  const float doubt = p.softmax ? 2.f * (1.f + EPL + 12.f) * 5.9604645e-8f : 4.7683716e-7f;
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    if (num[s] < 0) continue;
    const float l = key[s];
    const float sc = p.softmax ? (m == -inf ? 0.f : (l == m ? 1.f : expf(l - m)) * inv) : 1.f / (1.f + expf(-l));
    sv[num[s]] = sc;
    if (p.bias) {
      key[s] = sc + p.bias[num[s]];
      if (isnan(key[s])) key[s] = -inf;
    }
  }

  bool exactly = false;  // the whole row again in 64 bits
  int live = p.E;        // keys in the choice
  if (p.topk_group < p.n_group) {
    // group scores: P lanes a group
    const int size = p.E / p.n_group;
    const bool by_key = p.bias != nullptr || p.group_top == 1;
#pragma unroll
    for (int s = 0; s < EPL; ++s)
      if (num[s] >= 0) kv[num[s] + (num[s] >> 5)] = key[s];
    __syncwarp();
    int P = 32;
    while (32 / P < p.n_group) P >>= 1;
    const int g = lane / P, sub = lane & (P - 1);
    float b1 = -inf, b2 = -inf;
    if (g < p.n_group) {
      for (int j = sub; j < size; j += P) {
        const int i = g * size + j;
        top_two(b1, b2, by_key ? kv[i + (i >> 5)] : sv[i]);
      }
    }
    for (int d = 1; d < P; d <<= 1) {
      const float o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, d), o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, d);
      top_two(b1, b2, o1);
      top_two(b1, b2, o2);
    }
    float gs = p.group_top == 2 && size > 1 ? b1 + b2 : b1;
    if (isnan(gs)) gs = -inf;
    int rank = 0;
    for (int o = 0; o < p.n_group; ++o) {
      const float v = __shfl_sync(0xFFFFFFFFu, gs, o * P);
      rank += (v > gs || (v == gs && o < g)) ? 1 : 0;
    }
    const bool in = g < p.n_group && rank < p.topk_group;
    if (p.bias != nullptr || p.group_top == 2) {  // otherwise the scores are logits, and exact
      float lo = in ? gs : inf, hi = in || g >= p.n_group ? -inf : gs;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, off));
      }
      exactly = !(lo - hi > 2.f * doubt + 4.7683716e-7f * fmaxf(fabsf(lo), fabsf(hi))) && !(hi == -inf && lo > -inf);
    }
    const unsigned heads = __ballot_sync(0xFFFFFFFFu, in && sub == 0);
    if (in && sub == 0) chosen[__popc(heads & ((1u << lane) - 1u))] = g;
    __syncwarp();
    // the keys of the chosen groups, dealt out evenly again
    live = p.topk_group * size;
    const unsigned recip = ((1u << 20) + size - 1) / size;  // j / size for j < 1024
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      const int j = lane + 32 * s;
      num[s] = -1;
      key[s] = -inf;
      if (j < live) {
        const int q = static_cast<int>((static_cast<unsigned>(j) * recip) >> 20);
        num[s] = chosen[q] * size + (j - q * size);
        key[s] = kv[num[s] + (num[s] >> 5)];
      }
    }
  }

  int id = 0;
  float score = 0.f;
  int n = 0;
  if (!exactly) {
    // tau: the smallest of G >= k maxima over G groups of lanes is met by at
    // least k keys, so every one of the k best is >= tau; what may be as good
    // within the doubt is a candidate too
    float tau = key[0];
#pragma unroll
    for (int s = 1; s < EPL; ++s) tau = fmaxf(tau, key[s]);
    for (int d = 1; d < 32 && 32 / (2 * d) >= p.k; d <<= 1) tau = fmaxf(tau, __shfl_xor_sync(0xFFFFFFFFu, tau, d));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) tau = fminf(tau, __shfl_xor_sync(0xFFFFFFFFu, tau, off));
    const float lim = p.bias && tau > -inf ? tau - (doubt + 4.7683716e-7f * fabsf(tau)) : tau;
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      const bool take = num[s] >= 0 && key[s] >= lim;
      const unsigned bal = __ballot_sync(0xFFFFFFFFu, take);
      const int at = n + __popc(bal & ((1u << lane) - 1u));
      if (take && at < kCandidates) list[at] = candidate(key[s], num[s]);
      n += __popc(bal);
    }
    exactly = n > kCandidates;
  }
  if (!exactly) {
    // rank = how many candidates beat this one (they are all different)
    __syncwarp();
    for (int b = 0; b < n; b += 64) {
      const uint64_t v0 = b + lane < n ? list[b + lane] : ~0ull, v1 = b + lane + 32 < n ? list[b + lane + 32] : ~0ull;
      int r0 = 0, r1 = 0;
#pragma unroll 4
      for (int c = 0; c < n; ++c) {
        const uint64_t o = list[c];
        r0 += o > v0 ? 1 : 0;
        r1 += o > v1 ? 1 : 0;
      }
      if (b + lane < n && r0 <= p.k) best[r0] = v0;
      if (b + lane + 32 < n && r1 <= p.k) best[r1] = v1;
    }
    __syncwarp();
    const uint64_t mine = lane < p.k ? best[lane] : 0ull;
    id = lane < p.k ? candidate_expert(mine) : 0;
    if (p.bias) {
      bool close = false;
      if (lane < p.k && lane + 1 < n) {
        const uint64_t next = best[lane + 1];
        const float a = order_value(static_cast<uint32_t>(mine >> 32)), b = order_value(static_cast<uint32_t>(next >> 32));
        close = !(a - b > doubt + 4.7683716e-7f * fmaxf(fabsf(a), fabsf(b))) && !(b == -inf && a > -inf);
        if (close) {  // the same logit and bias are a tie in any precision
          const int o = candidate_expert(next);
          close = row[id] != row[o] || p.bias[id] != p.bias[o];
        }
      }
      if (__any_sync(0xFFFFFFFFu, close)) {
        if (p.softmax) {
          exactly = true;
        } else {
          // the candidates again in 64 bits: value v, ties to the lower expert
          double* exact = reinterpret_cast<double*>(list);
          const int per = (n + 31) / 32;
          for (int c = 0; c < per; ++c) {
            const int at = c * 32 + lane;
            int e = -1;
            double v = 0.0;
            if (at < n) {
              e = candidate_expert(list[at]);
              const double z = isnan(row[e]) ? -__longlong_as_double(0x7FF0000000000000ll) : static_cast<double>(row[e]);
              v = 1.0 / (1.0 + exp(-z)) + static_cast<double>(p.bias[e]);
              if (isnan(v)) v = __longlong_as_double(0xFFF0000000000000ll);
            }
            __syncwarp();
            if (at < n) {
              exact[at] = v;
              reinterpret_cast<int*>(kv)[at] = e;
            }
          }
          __syncwarp();
          for (int c = 0; c < per; ++c) {
            const int at = c * 32 + lane;
            if (at >= n) continue;
            const double v = exact[at];
            const int e = reinterpret_cast<int*>(kv)[at];
            int r = 0;
            for (int o = 0; o < n; ++o) {
              const double u = exact[o];
              r += (u > v || (u == v && reinterpret_cast<int*>(kv)[o] < e)) ? 1 : 0;
            }
            if (r < p.k) chosen[r] = e;
          }
          __syncwarp();
          if (lane < p.k) id = chosen[lane];
        }
      }
    }
  }
  if (exactly) {
    double s64;
    __syncwarp();
    group_select_f64(p, row, reinterpret_cast<double*>(mem), reinterpret_cast<double*>(mem) + p.E, id, s64);
    score = static_cast<float>(s64);
  } else {
    score = lane < p.k ? sv[id] : 0.f;
  }
  float w = lane < p.k ? score : 0.f;
  if (p.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = id;
    p.w[t * p.k + lane] = p.scale * w;
  }
}

template <int EPL>
static cudaError_t launch_group_route(const GroupRouteParams& p, cudaStream_t stream) {
  const int smem = kGroupRouteWarps * route_smem(p.E);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(group_route_kernel<EPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T + kGroupRouteWarps - 1) / kGroupRouteWarps), 1, 1);
  cfg.blockDim = dim3(kGroupRouteWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, group_route_kernel<EPL>, p);
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
  cudaError_t e;
  if (E <= 32) e = launch_group_route<1>(p, stream);
  else if (E <= 64) e = launch_group_route<2>(p, stream);
  else if (E <= 128) e = launch_group_route<4>(p, stream);
  else if (E <= 256) e = launch_group_route<8>(p, stream);
  else if (E <= 512) e = launch_group_route<16>(p, stream);
  else e = launch_group_route<32>(p, stream);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

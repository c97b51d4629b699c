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
// instructions (two thirds of the cycles issue one); the data is 4 E bytes a
// token.  E = 256 in 8 groups, sigmoid with a bias: T = 1 3.2 us, T = 8192
// 12.6 us.
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

// Order-preserving keys of numbers (NaN counts as -inf; -0 and +0 share one).
// Every key is above 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u << 1) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t order_key64(double d) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(d));
  if ((u << 1) > 0xFFE0000000000000ull) u = 0xFFF0000000000000ull;
  if ((u << 1) == 0u) u = 0u;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// A logit with NaN as -inf.
__device__ __forceinline__ float logit(float l) { return isnan(l) ? __int_as_float(0xFF800000) : l; }

__device__ __forceinline__ double sigmoid_f64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// The choice of one token in 64 bits.  `sc` and `key` are E values each of
// this warp's shared memory.  Lane j < k gets the j-th id and its logit.  The
// 64-bit pipe is narrow, so it computes the values, and their integer keys are
// compared.
__device__ __noinline__ void group_select_f64(const GroupRouteParams& p, const float* __restrict__ row, double* sc,
                                              uint64_t* key, int& id, float& l) {
  const int lane = threadIdx.x & 31;
  const double inf = __longlong_as_double(0x7FF0000000000000ll);
  double m = -inf, sum = 1.0;
  if (p.softmax) {
    for (int i = lane; i < p.E; i += 32) m = fmax(m, static_cast<double>(logit(row[i])));
    m = warp_max_f64(m);
    double part = 0.0;
    for (int i = lane; i < p.E; i += 32) {
      const double z = logit(row[i]);
      const double e = m == -inf ? 0.0 : z == m ? 1.0 : exp(z - m);
      sc[i] = e;
      part += e;
    }
    sum = warp_sum_f64(part);
    if (sum == 0.0) sum = 1.0;
  }
  const int size = p.E / p.n_group;
  const bool grouped = p.topk_group < p.n_group;
  for (int i = lane; i < p.E; i += 32) {
    const float l = logit(row[i]);
    const double s = p.softmax ? sc[i] / sum : sigmoid_f64(l);
    sc[i] = s;
    key[i] = order_key64(p.bias ? s + static_cast<double>(p.bias[i]) : static_cast<double>(l));
  }
  __syncwarp();
  if (grouped) {
    // group scores; the keys of the groups that do not stay become 0
    double gs = -inf;
    if (lane < p.n_group) {
      uint64_t k1 = 0, k2 = 0;
      int i1 = -1, i2 = -1;
      for (int i = lane * size; i < (lane + 1) * size; ++i) {
        // without a bias the scores order like the logits, whose keys these are
        const uint64_t v = key[i];
        if (v > k1) { k2 = k1; i2 = i1; k1 = v; i1 = i; }
        else if (v > k2) { k2 = v; i2 = i; }
      }
      const bool by_logit = !p.bias && p.group_top == 1;
      auto value = [&](int i) {
        return by_logit ? static_cast<double>(logit(row[i])) : sc[i] + (p.bias ? static_cast<double>(p.bias[i]) : 0.0);
      };
      gs = value(i1);
      if (p.group_top == 2 && size > 1) gs += value(i2);
    }
    const uint64_t gk = lane < p.n_group ? order_key64(gs) : 0ull;
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const uint64_t o = __shfl_sync(0xFFFFFFFFu, gk, g);
      rank += (o > gk || (o == gk && g < lane)) ? 1 : 0;
    }
    const unsigned in = __ballot_sync(0xFFFFFFFFu, lane < p.n_group && rank < p.topk_group);
    for (int i = lane; i < p.E; i += 32)
      if (!((in >> (i / size)) & 1u)) key[i] = 0ull;
    __syncwarp();
  }
  // k rounds: the largest key, the lowest expert among equals
  id = 0;
  for (int r = 0; r < p.k; ++r) {
    uint64_t b = 0ull;
    int at = 0x7FFFFFFF;
    for (int i = lane; i < p.E; i += 32) {
      const uint64_t v = key[i];
      if (v > b) { b = v; at = i; }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const uint64_t ob = __shfl_xor_sync(0xFFFFFFFFu, b, off);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, off);
      if (ob > b || (ob == b && oa < at)) { b = ob; at = oa; }
    }
    if (lane == r) id = at;
    __syncwarp();
    if (lane == 0) key[at] = 0ull;
    __syncwarp();
  }
  l = logit(row[id]);
}

// Adds v to the two largest values b1 >= b2 so far.
__device__ __forceinline__ void top_two(float& b1, float& b2, float v) {
  b2 = fmaxf(b2, fminf(b1, v));
  b1 = fmaxf(b1, v);
}

// A candidate: a larger value is the better choice (larger key, then lower
// expert).
__device__ __forceinline__ uint64_t candidate(float v, int expert) {
  return (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(0xFFFFFFFFu - static_cast<uint32_t>(expert));
}
__device__ __forceinline__ int candidate_expert(uint64_t c) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(c));
}

// Whether a >= b may be in the wrong order.  The error of a choice value is
// `doubt` / 2 and one rounding of its size.
__device__ __forceinline__ bool too_close(float a, float b, float doubt) {
  const float inf = __int_as_float(0x7F800000);
  return !(a - b > doubt + 4.7683716e-7f * fmaxf(fabsf(a), fabsf(b))) && !(b == -inf && a > -inf);
}

// Smallest and largest of the warp's values.
__device__ __forceinline__ float warp_least(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_most(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

// The score of a chosen logit l (-inf: none) in a row with small ones, m and
// inv the softmax' maximum and 1 / sum.  Divided by their sum, only the scores'
// ratios count: where the best chosen score is below e^-16 they are taken
// relative to it, as scores of 32 bits end at e^-103 (and 1 / (1 + expf(-l)) at
// e^-88).  A score below 2^-1022 counts as 0.
template <bool SOFTMAX>
__device__ __forceinline__ float small_weight(float l, float m, float inv, int renorm) {
  const float inf = __int_as_float(0x7F800000), ref = SOFTMAX ? m : 0.f;
  const float top = renorm ? warp_most(l) : inf;
  if (top - ref < -16.f) return l - ref < -708.39642f ? 0.f : expf(l - top) / (SOFTMAX ? 1.f : 1.f + expf(l));
  if (SOFTMAX) return m == -inf ? 0.f : (l == m ? 1.f : expf(l - m)) * inv;
  return l < -80.f ? expf(l) / (1.f + expf(l)) : 1.f / (1.f + expf(-l));
}

// Shared memory of one warp, in bytes: the larger of the 32-bit selection's
// arrays and the 64-bit one's.
__host__ __device__ constexpr int route_list_at(int E) { return (E * 4 + (E + E / 32 + 1) * 4 + 15) / 16 * 16; }
__host__ __device__ constexpr int route_smem(int E) {
  const int fast = route_list_at(E) + (kCandidates + 8 + 40) * 8 + 128 + kCandidates * 4, slow = E * 16;
  return (fast > slow ? fast : slow) / 16 * 16 + 16;
}

// SOFTMAX, BIAS, GROUPS: which steps the call needs.
template <int EPL, bool SOFTMAX, bool BIAS, bool GROUPS>
__global__ void __launch_bounds__(kGroupRouteWarps * 32) group_route_kernel(const GroupRouteParams p) {
  extern __shared__ __align__(16) uint8_t route_mem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGroupRouteWarps + warp;
  const float inf = __int_as_float(0x7F800000);
  uint8_t* mem = route_mem + static_cast<size_t>(warp) * route_smem(p.E);
  float* lv = reinterpret_cast<float*>(mem);         // [E] logits
  float* kv = lv + p.E;                              // [E + E / 32] choice values, one word of padding per 32
  uint64_t* list = reinterpret_cast<uint64_t*>(mem + route_list_at(p.E));
  uint64_t* best = list + kCandidates + 8;           // [k + 1]
  int* chosen = reinterpret_cast<int*>(best + 40);   // [32] groups that stay
  int* who = chosen + 32;                            // [kCandidates] experts compared in 64 bits
  const float* row = p.logits + t * p.E;
  allow_dependent_launch();
  // the bias is a parameter, but it too is read after the wait: a balancing
  // step may just have written it
  grid_dependency_wait();
  if (t >= p.T) return;

  float key[EPL], bias[BIAS ? EPL : 1];
  int num[EPL];  // the expert of each key; -1: none
  float m = -inf;
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    const int i = lane + 32 * s;
    num[s] = i < p.E ? i : -1;
    key[s] = i < p.E ? row[i] : -inf;
    if (BIAS) bias[s] = i < p.E ? p.bias[i] : 0.f;
  }
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    key[s] = logit(key[s]);
    if (SOFTMAX) m = fmaxf(m, key[s]);
    if (num[s] >= 0) lv[num[s]] = key[s];
  }
  // Choice values from the short exponential and quotient.  A sigmoid: the
  // exponential within 2^-21 + 2^-24 |l| of itself, which moves s by s (1 - s)
  // of that (s (1 - s) <= 1/4, times |l| <= 0.23), and the sum and quotient
  // 5 * 2^-24: together under 2^-21.  A softmax term: 2^-21 + 2^-23 |l - m| of
  // itself, s |l - m| < 1/2, the sum of E terms and the quotient (E / 32 + 12)
  // 2^-24.  Two values: twice that.
  const float doubt = SOFTMAX ? 2.f * (8.f + 1.f + EPL + 12.f) * 5.9604645e-8f : 9.536743e-7f;
  float inv = 1.f;
  if (SOFTMAX) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  }
  // Softmax terms, for the choice and for the weights' sum: expf where the
  // weights depend on them.
  float e[SOFTMAX ? EPL : 1];
  if (SOFTMAX) {
    float z = 0.f;
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      e[s] = m == -inf || num[s] < 0 ? 0.f : key[s] == m ? 1.f : expf(key[s] - m);
      z += e[s];
    }
    z = warp_sum(z);
    inv = z > 0.f ? 1.f / z : 0.f;
  }
  if (BIAS) {
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      const float sc = SOFTMAX ? e[s] * inv : __fdividef(1.f, 1.f + __expf(fminf(-key[s], 80.f)));
      key[s] = sc + bias[s];
      if (num[s] < 0 || isnan(key[s])) key[s] = -inf;
    }
  }

  bool exactly = false;  // the whole row again in 64 bits
  int live = p.E;        // keys in the choice
  if (GROUPS) {
    // group scores: P lanes a group
    const int size = p.E / p.n_group;
    const bool by_key = BIAS || p.group_top == 1;
#pragma unroll
    for (int s = 0; s < EPL; ++s)
      if (num[s] >= 0) kv[num[s] + (num[s] >> 5)] = key[s];
    __syncwarp();
    int P = 32;
    while (32 / P < p.n_group) P >>= 1;
    const int g = lane / P, sub = lane & (P - 1);
    float b1 = -inf, b2 = -inf;
    if (g < p.n_group) {
#pragma unroll 4
      for (int j = sub; j < size; j += P) {
        const int i = g * size + j;
        top_two(b1, b2, kv[i + (i >> 5)]);
      }
    }
    for (int d = 1; d < P; d <<= 1) {
      const float o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, d), o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, d);
      top_two(b1, b2, o1);
      top_two(b1, b2, o2);
    }
    const bool two = p.group_top == 2 && size > 1;
    if (!by_key) {  // without a bias the best logits have the best scores
      b1 = SOFTMAX ? (m == -inf ? 0.f : (b1 == m ? 1.f : expf(b1 - m)) * inv) : 1.f / (1.f + expf(-b1));
      b2 = SOFTMAX ? (m == -inf ? 0.f : (b2 == m ? 1.f : expf(b2 - m)) * inv) : 1.f / (1.f + expf(-b2));
    }
    float gs = two ? b1 + b2 : b1;
    if (isnan(gs)) gs = -inf;
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < p.n_group; ++o) {
      const float v = __shfl_sync(0xFFFFFFFFu, gs, o * P);
      rank += (v > gs || (v == gs && o < g)) ? 1 : 0;
    }
    bool in = g < p.n_group && rank < p.topk_group;
    if (BIAS || p.group_top == 2) {  // otherwise the scores are logits, and exact
      // A group's score is as uncertain as its values, whose roundings go by
      // their own size (they may cancel in the sum): twice doubt / 2 and 2^-24
      // of each value and of the sum.  A sum at the end of the range may
      // stand for anything beyond it.
      const float big = 3.4028235e38f;
      const float err = doubt + 2.3841858e-7f * (fabsf(b1) + (two ? fabsf(b2) : 0.f));
      const float low = gs == inf ? big : gs == -inf ? -inf : gs - err, high = gs == -inf ? -big : gs == inf ? inf : gs + err;
      const bool group = g < p.n_group, stays = group && rank < p.topk_group;
      const float lo = warp_least(stays ? low : inf), hi = warp_most(group && !stays ? high : -inf);
      if (!(lo > hi)) {
        if (SOFTMAX || !BIAS) {
          exactly = true;
        } else {
          // the values that may be among a group's best, again in 64 bits
          const float need = two ? b2 : b1;
          const float lim = fabsf(need) < inf ? need - (doubt + 4.7683716e-7f * fabsf(need)) : need;
          int n = 0;
          for (int j = 0; j < (size + P - 1) / P; ++j) {
            const int i = g * size + j * P + sub;
            const bool take = g < p.n_group && j * P + sub < size && kv[i + (i >> 5)] >= lim;
            const unsigned bal = __ballot_sync(0xFFFFFFFFu, take);
            const int at = n + __popc(bal & ((1u << lane) - 1u));
            if (take && at < kCandidates) who[at] = i;
            n += __popc(bal);
          }
          exactly = n > kCandidates;
          if (!exactly) {
            __syncwarp();
            double* val = reinterpret_cast<double*>(list);
            for (int at = lane; at < n; at += 32) val[at] = sigmoid_f64(lv[who[at]]) + static_cast<double>(p.bias[who[at]]);
            __syncwarp();
            uint64_t k1 = 0, k2 = 0;
            double v1 = 0.0, v2 = 0.0;
            for (int at = 0; at < n; ++at) {
              const unsigned d = static_cast<unsigned>(who[at] - g * size);
              if (d < static_cast<unsigned>(size)) {
                const double v = val[at];
                const uint64_t k = order_key64(v);
                if (k > k1) { k2 = k1; v2 = v1; k1 = k; v1 = v; }
                else if (k > k2) { k2 = k; v2 = v; }
              }
            }
            const uint64_t gk = g < p.n_group ? order_key64(two ? v1 + v2 : v1) : 0ull;
            rank = 0;
            for (int o = 0; o < p.n_group; ++o) {
              const uint64_t v = __shfl_sync(0xFFFFFFFFu, gk, o * P);
              rank += (v > gk || (v == gk && o < g)) ? 1 : 0;
            }
            in = g < p.n_group && rank < p.topk_group;
          }
        }
      }
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
      if (32 * s >= live) continue;  // (the same for all lanes)
      if (j < live) {
        const int q = static_cast<int>((static_cast<unsigned>(j) * recip) >> 20);
        num[s] = chosen[q] * size + (j - q * size);
        key[s] = kv[num[s] + (num[s] >> 5)];
      }
    }
  }

  int id = 0;
  int n = 0;
  if (!exactly) {
    // tau: the smallest of G >= k maxima over G groups of lanes is met by at
    // least k keys, so every one of the k best is >= tau (places without an
    // expert hold -inf and are in no group's way); what may be as good within
    // the doubt is a candidate too.  An infinite tau is exact.
    float tau = key[0];
#pragma unroll
    for (int s = 1; s < EPL; ++s) tau = fmaxf(tau, key[s]);
    for (int d = 1; d < 32 && 32 / (2 * d) >= p.k; d <<= 1) tau = fmaxf(tau, __shfl_xor_sync(0xFFFFFFFFu, tau, d));
    tau = order_value(__reduce_min_sync(0xFFFFFFFFu, order_key(tau)));
    const float lim = BIAS && fabsf(tau) < inf ? tau - (doubt + 4.7683716e-7f * fabsf(tau)) : tau;
    unsigned bal[EPL];
#pragma unroll
    for (int s = 0; s < EPL; ++s)
      bal[s] = !GROUPS || 32 * s < live ? __ballot_sync(0xFFFFFFFFu, num[s] >= 0 && key[s] >= lim) : 0u;
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      if (GROUPS && 32 * s >= live) break;
      const int at = n + __popc(bal[s] & ((1u << lane) - 1u));
      if (((bal[s] >> lane) & 1u) && at < kCandidates) list[at] = candidate(key[s], num[s]);
      n += __popc(bal[s]);
    }
    exactly = n > kCandidates;
  }
  if (!exactly) {
    // rank = how many candidates beat this one (they are all different); the
    // list is padded with 0, below every candidate, to whole blocks of 8
    const int blocks = (n + 7) >> 3;
    if (lane < 8 * blocks - n) list[n + lane] = 0ull;
    __syncwarp();
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(list);
    for (int b = 0; b < n; b += 32) {  // usually one round
      const uint64_t v = b + lane < n ? list[b + lane] : ~0ull;
      int r = 0;
      for (int c = 0; c < blocks; ++c) {
        ulonglong2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pairs[4 * c + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) r += (o[i].x > v ? 1 : 0) + (o[i].y > v ? 1 : 0);
      }
      if (b + lane < n && r <= p.k) best[r] = v;
    }
    __syncwarp();
    const uint64_t mine = lane < p.k ? best[lane] : 0ull;
    id = lane < p.k ? candidate_expert(mine) : 0;
    if (BIAS) {
      // the same logit and bias are a tie in any precision
      auto doubtful = [&](uint64_t better, uint64_t worse) {
        return too_close(order_value(static_cast<uint32_t>(better >> 32)), order_value(static_cast<uint32_t>(worse >> 32)),
                         doubt);
      };
      auto equal = [&](int x, int y) { return lv[x] == lv[y] && p.bias[x] == p.bias[y]; };
      bool close = false, tied = false;
      if (lane < p.k && lane + 1 < n) {
        const uint64_t next = best[lane + 1];
        close = doubtful(mine, next);
        if (close && equal(id, candidate_expert(next))) {
          close = false;
          tied = lane == p.k - 1;
        }
      }
      if (__any_sync(0xFFFFFFFFu, tied)) {
        // behind those equal to the last one chosen may stand one that only 64
        // bits tell from them
        const uint64_t last = best[p.k - 1];
        for (int at = lane; at < n; at += 32) {
          const uint64_t v = list[at];
          if (v < last && doubtful(last, v) && !equal(candidate_expert(last), candidate_expert(v))) close = true;
        }
      }
      if (__any_sync(0xFFFFFFFFu, close)) {
        if (SOFTMAX) {
          exactly = true;
        } else {
          // the candidates again in 64 bits
          for (int at = lane; at < n; at += 32) {
            const int x = candidate_expert(list[at]);
            who[at] = x;
            list[at] = order_key64(sigmoid_f64(lv[x]) + static_cast<double>(p.bias[x]));
          }
          __syncwarp();
          for (int at = lane; at < n; at += 32) {
            const uint64_t v = list[at];
            const int x = who[at];
            int r = 0;
            for (int o = 0; o < n; ++o) {
              const uint64_t u = list[o];
              r += (u > v || (u == v && who[o] < x)) ? 1 : 0;
            }
            if (r < p.k) best[r] = static_cast<uint64_t>(x);
          }
          __syncwarp();
          if (lane < p.k) id = static_cast<int>(best[lane]);
        }
      }
    }
  }
  float l = lv[id];
  if (exactly) {
    __syncwarp();
    group_select_f64(p, row, reinterpret_cast<double*>(mem), reinterpret_cast<uint64_t*>(mem) + p.E, id, l);
  }
  if (lane >= p.k) l = -inf;
  // The weights, the same way whatever made the choice.
  float w = 0.f;
  if (lane < p.k) w = SOFTMAX ? (m == -inf ? 0.f : (l == m ? 1.f : expf(l - m)) * inv) : 1.f / (1.f + expf(-l));
  if (__any_sync(0xFFFFFFFFu, lane < p.k && l - (SOFTMAX ? m : 0.f) < -16.f)) w = small_weight<SOFTMAX>(l, m, inv, p.renorm);
  if (p.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = id;
    p.w[t * p.k + lane] = p.scale * w;
  }
}

template <int EPL, bool SOFTMAX, bool BIAS, bool GROUPS>
static cudaError_t launch_group_route(const GroupRouteParams& p, cudaStream_t stream) {
  const int smem = kGroupRouteWarps * route_smem(p.E);
  const auto kernel = group_route_kernel<EPL, SOFTMAX, BIAS, GROUPS>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int EPL>
static cudaError_t launch_group_route(const GroupRouteParams& p, cudaStream_t stream) {
  const bool g = p.topk_group < p.n_group;
  if (p.softmax) {
    if (p.bias) return g ? launch_group_route<EPL, true, true, true>(p, stream) : launch_group_route<EPL, true, true, false>(p, stream);
    return g ? launch_group_route<EPL, true, false, true>(p, stream) : launch_group_route<EPL, true, false, false>(p, stream);
  }
  if (p.bias) return g ? launch_group_route<EPL, false, true, true>(p, stream) : launch_group_route<EPL, false, true, false>(p, stream);
  return g ? launch_group_route<EPL, false, false, true>(p, stream) : launch_group_route<EPL, false, false, false>(p, stream);
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
  if (E <= 64) e = launch_group_route<2>(p, stream);
  else if (E <= 128) e = launch_group_route<4>(p, stream);
  else if (E <= 256) e = launch_group_route<8>(p, stream);
  else e = launch_group_route<32>(p, stream);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

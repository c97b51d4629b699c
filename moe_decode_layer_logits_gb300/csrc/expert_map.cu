// moe_expert_map: the expert-sorted row layout of a routed batch (stable
// counting sort of the T * k slots by expert, tokens ascending in each).
#include "host_util.h"
#include "common.cuh"

namespace moe {

struct ExpertMapParams {
  const int32_t* ids;
  int32_t* row_map;
  int32_t* row_token;
  int32_t* offsets;
  int32_t* counts;
  int64_t n_rows;
  int64_t slots;  // T * k
  int E, k, block;
};

constexpr int kMapThreads = 1024;

// One CTA: counts, offsets, then one warp per expert places its slots in
// ascending order.
__global__ void __launch_bounds__(kMapThreads) expert_map_kernel(const ExpertMapParams p) {
  __shared__ int count_s[MOE_MAX_E];
  __shared__ int start_s[MOE_MAX_E + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  grid_dependency_wait();
  for (int e = tid; e < p.E; e += kMapThreads) count_s[e] = 0;
  __syncthreads();
  for (int64_t i = tid; i < p.slots; i += kMapThreads) {
    const int e = p.ids[i];
    if (e >= 0 && e < p.E) atomicAdd(&count_s[e], 1);
    else p.row_map[i] = -1;
  }
  for (int64_t i = tid; i < p.n_rows; i += kMapThreads) p.row_token[i] = -1;
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    for (int e = 0; e < p.E; ++e) {
      start_s[e] = at;
      at += (count_s[e] + p.block - 1) / p.block * p.block;
    }
    start_s[p.E] = at;
  }
  __syncthreads();
  for (int e = tid; e <= p.E; e += kMapThreads) {
    p.offsets[e] = start_s[e];
    if (e < p.E) p.counts[e] = count_s[e];
  }
  for (int e = warp; e < p.E; e += kMapThreads / 32) {
    int at = start_s[e];
    for (int64_t b = 0; b < p.slots; b += 32) {
      const int64_t i = b + lane;
      const bool mine = i < p.slots && p.ids[i] == e;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) {
        const int row = at + __popc(m & ((1u << lane) - 1u));
        p.row_map[i] = row;
        p.row_token[row] = static_cast<int>(i / p.k);
      }
      at += __popc(m);
    }
  }
}

}  // namespace moe

extern "C" int64_t moe_expert_rows(int64_t T, int64_t E, int32_t k, int32_t block) {
  if (T < 0 || E < 1 || k < 1 || block < 1 || T > (static_cast<int64_t>(1) << 31) / k) return -1;
  const int64_t n = T * k;
  return n + (n < E ? n : E) * (block - 1);
}

extern "C" int moe_expert_map(const int32_t* topk_ids, int32_t* row_map, int32_t* row_token, int32_t* offsets,
                              int32_t* counts, int64_t n_rows, int64_t T, int64_t E, int32_t k, int32_t block,
                              cudaStream_t stream) {
  using namespace moe;
  if (T < 0 || E < 1 || k < 1 || k > MOE_MAX_K || block < 1) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_E || block > 4096 || T > (static_cast<int64_t>(1) << 30) / k || n_rows > 0x7FFFFFFFll)
    return MOE_ERR_UNSUPPORTED;
  if (n_rows < moe_expert_rows(T, E, k, block)) return MOE_ERR_INVALID_ARG;
  if (!offsets || !counts || (T > 0 && (!topk_ids || !row_map)) || (n_rows > 0 && !row_token))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(row_map, 4) || !aligned(row_token, 4) || !aligned(offsets, 4) ||
      !aligned(counts, 4))
    return MOE_ERR_MISALIGNED;
  ExpertMapParams p{topk_ids, row_map, row_token, offsets, counts, n_rows, T * k, static_cast<int>(E), k, block};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kMapThreads, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, expert_map_kernel, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

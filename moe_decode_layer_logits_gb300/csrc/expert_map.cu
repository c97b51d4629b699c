// moe_expert_map: the expert-sorted row layout of a routed batch, a stable
// counting sort of the T * k slots by expert (tokens ascending in each).
//
// One launch of one thread-block cluster (a single CTA for small batches), no
// global scratch: CTA r takes the r-th stretch of the slots, each of its warps
// a stretch of that.  Every warp counts its slots per expert in shared memory;
// the counts are added up over the warps and, through distributed shared
// memory, over the cluster, and scanned over the experts; then each warp walks
// its slots once more, 32 at a time and in order, and gives every slot its
// place (equal experts within the 32 by ballots on the bits of the expert).  Integer counts only:
// the layout does not depend on the order of the atomics.  Bound by latency:
// two passes over a warp's slots and two cluster barriers; more warps shorten
// the walks until adding up their counts costs as much.
#include "expert_map.h"
#include "host_util.h"
#include "common.cuh"

namespace moe {

constexpr int kMapMaxWarps = 32;
constexpr int kMapBatch = 8;  // groups of 32 slots whose ids a warp loads at once
constexpr int kMapMaxCluster = 8;

// Shared memory: [warps][E] counts, then places; [E] each: this CTA's counts,
// the cluster's, this CTA's first row.
static size_t map_smem(int warps, int E) { return static_cast<size_t>(warps + 3) * E * sizeof(int); }

__global__ void __launch_bounds__(kMapMaxWarps * 32) expert_map_kernel(const ExpertMapParams p) {
  extern __shared__ int map_mem[];
  __shared__ int warp_rows[kMapMaxWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5, E = p.E;
  int* hist = map_mem;
  int* mine = map_mem + W * E;
  int* total = mine + E;
  int* first = total + E;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  allow_dependent_launch();
  for (int i = tid; i < W * E; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  grid_dependency_wait();

  // rows that no slot has stay -1: every row is filled before the cluster
  // barrier, and the places are written after it
  {
    const int64_t threads = static_cast<int64_t>(C) * blockDim.x, at = static_cast<int64_t>(rank) * blockDim.x + tid;
    const int64_t quads = (reinterpret_cast<uintptr_t>(p.row_token) & 15) == 0 ? p.n_rows / 4 : 0;
    for (int64_t i = at; i < quads; i += threads) reinterpret_cast<int4*>(p.row_token)[i] = make_int4(-1, -1, -1, -1);
    for (int64_t i = quads * 4 + at; i < p.n_rows; i += threads) p.row_token[i] = -1;
  }
  // this warp's slots, whole groups of 32
  const int64_t groups = (p.slots + 31) / 32, walkers = static_cast<int64_t>(C) * W;
  const int64_t me = static_cast<int64_t>(rank) * W + warp;
  const int64_t beg = groups * me / walkers * 32, end = min(p.slots, groups * (me + 1) / walkers * 32);
  int* count = hist + warp * E;
  int id[kMapBatch];
  auto load = [&](int64_t g) {  // ids of the groups from slot g; E where there is none
#pragma unroll
    for (int b = 0; b < kMapBatch; ++b) {
      const int64_t i = g + b * 32 + lane;
      const int e = i < end ? p.ids[i] : -1;
      id[b] = e >= 0 && e < E - p.rest ? e : E;
      if (p.rest && i < end && id[b] == E) {
        if (e >= 0 && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
        id[b] = E - 1;
      }
    }
  };
  for (int64_t g = beg; g < end; g += 32 * kMapBatch) {
    load(g);
#pragma unroll
    for (int b = 0; b < kMapBatch; ++b)
      if (id[b] < E) atomicAdd(&count[id[b]], 1);
  }
  __syncthreads();
  // over the warps: places before each warp, and this CTA's counts; `parts`
  // neighbouring threads share an expert
  int parts = 1;
  while (parts * 2 * E <= static_cast<int>(blockDim.x) && parts * 2 <= W) parts *= 2;
  const int q = tid & (parts - 1), span = (W + parts - 1) / parts, w0 = min(W, q * span), w1 = min(W, w0 + span);
  for (int e0 = 0; e0 < E; e0 += blockDim.x / parts) {
    const int e = e0 + tid / parts;
    int sum = 0;
    if (e < E)
      for (int w = w0; w < w1; ++w) sum += hist[w * E + e];
    int at = sum;
    for (int off = 1; off < parts; off <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, at, off, parts);
      if (q >= off) at += v;
    }
    if (e < E) {
      if (q == parts - 1) mine[e] = at;
      at -= sum;
      for (int w = w0; w < w1; ++w) {
        const int c = hist[w * E + e];
        hist[w * E + e] = at;
        at += c;
      }
    }
  }
  cluster_arrive_release();
  cluster_wait_acquire();
  // over the cluster, then over the experts (thread i: `per` neighbours)
  const int per = (E + blockDim.x - 1) / blockDim.x;
  const int eb = min(E, tid * per), ee = min(E, eb + per);
  int rows = 0;
  for (int e = eb; e < ee; ++e) {
    int before = 0, all = 0;
    int c[kMapMaxCluster];
#pragma unroll
    for (int r = 0; r < kMapMaxCluster; ++r) c[r] = r < C ? *cluster.map_shared_rank(&mine[e], r) : 0;
#pragma unroll
    for (int r = 0; r < kMapMaxCluster; ++r) {
      if (r < rank) before += c[r];
      all += c[r];
    }
    first[e] = before;
    total[e] = all;
    rows += (all + p.block - 1) / p.block * p.block;
    if (rank == 0) p.counts[e] = all;
  }
  int upto = rows;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) warp_rows[warp] = upto;
  cluster_arrive_release();  // this CTA has read its peers' counts
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += warp_rows[w];
  base += upto - rows;
  for (int e = eb; e < ee; ++e) {
    first[e] += base;
    if (rank == 0) p.offsets[e] = base;
    base += (total[e] + p.block - 1) / p.block * p.block;
  }
  if (tid == static_cast<int>(blockDim.x) - 1 && rank == 0) p.offsets[E] = base;
  __syncthreads();
  // places
  const int bits = 32 - __clz(E);
  for (int64_t g = beg; g < end; g += 32 * kMapBatch) {
    if (end - beg > 32 * kMapBatch) load(g);  // otherwise they are still there
#pragma unroll
    for (int b = 0; b < kMapBatch; ++b) {
      if (g + b * 32 >= end) break;
      const int64_t i = g + b * 32 + lane;
      const int e = id[b];
      unsigned same = 0xFFFFFFFFu;  // lanes with this lane's expert
      for (int bit = 0; bit < bits; ++bit) {
        const unsigned set = __ballot_sync(0xFFFFFFFFu, (e >> bit) & 1);
        same &= (e >> bit) & 1 ? set : ~set;
      }
      const int before = __popc(same & ((1u << lane) - 1u));
      int row = -1;
      if (e < E) row = count[e] + before;
      __syncwarp();
      if (e < E && before == 0) count[e] = row + __popc(same);
      __syncwarp();
      if (e < E) {
        row += first[e];
        p.row_token[row] = static_cast<int>(i) / p.k;
      }
      if (i < end && p.row_map) p.row_map[i] = row;
    }
  }
  cluster_wait_acquire();  // no CTA leaves while a peer may read its counts
}

cudaError_t launch_expert_map(const ExpertMapParams& p, cudaStream_t stream) {
  // A warp for about 128 slots or 1024 rows.  Small CTAs have the shorter
  // barriers, so the cluster grows first (8 warps each up to 8 CTAs), then the
  // CTAs, up to 32 warps.  With 8 / 16 / 32 warps a CTA at E = 256, k = 8:
  // T = 512 5.1 / 6.0 / 8.7 us, T = 4096 10.4 / 8.2 / 9.6 us, T = 32768
  // 59 / 39 / 33 us.
  int64_t want = (p.slots + 127) / 128;
  if (want < (p.n_rows + 1023) / 1024) want = (p.n_rows + 1023) / 1024;
  int C = 1;
  while (C < kMapMaxCluster && static_cast<int64_t>(C) * 8 < want) C *= 2;
  const int64_t per_cta = (want + C - 1) / C;
  const int warps = per_cta < 8 ? 8 : per_cta > kMapMaxWarps ? kMapMaxWarps : static_cast<int>(per_cta);
  const size_t smem = map_smem(warps, p.E);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(expert_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(map_smem(kMapMaxWarps, MOE_MAX_E + 1)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(warps * 32), 1, 1);
  cfg.dynamicSmemBytes = launch_smem(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, expert_map_kernel, p);
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
  const ExpertMapParams p{topk_ids, row_map, row_token, offsets, counts, n_rows, T * k, static_cast<int>(E), k, block,
                          0, nullptr};
  if (launch_expert_map(p, stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

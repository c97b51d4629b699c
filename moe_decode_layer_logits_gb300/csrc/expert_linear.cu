// moe_expert_linear: the products of the routed rows with their experts'
// weights, out[r] = act(W_e x[src(r)]) for the rows r of expert e's segment;
// moe_adapter_linear: one shared projection with each token's low-rank
// adapter, out[t] = act(W x[t] + s_a B_a (A_a x[t])).
//
// FP32 sums of exact BF16 products; the activation works on the FP32 sums and
// the result is rounded to BF16 once.
#include "expert_gemm.h"
#include "host_util.h"
#include "common.cuh"

namespace moe {

struct LinearParams {
  const uint16_t* x;
  const int32_t* row_token;  // null: row r reads x[r]
  const uint16_t* w;
  const int32_t* offsets;  // null: one segment of n_rows rows
  const int32_t* counts;
  uint16_t* out;
  int64_t n_x, n_rows, N, K;
  int32_t* err_flag;
  // adapters
  const float* low;  // [T, R] scaled A x
  const uint16_t* b;
  const int32_t* ids;
  int R, L;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// 16 x 16 threads, a tile of 16 rows x 16 outputs.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) linear_kernel(const LinearParams p) {
  __shared__ float xs[16][33], ws[16][33], us[16][33];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int e = blockIdx.y;
  allow_dependent_launch();
  grid_dependency_wait();
  int64_t beg = 0, cnt = p.n_rows;
  if (p.offsets) {
    beg = p.offsets[e];
    cnt = p.counts[e];
    if (beg < 0 || cnt < 0 || beg + cnt > p.n_rows) {  // not a segment of the rows: skipped
      if (threadIdx.x == 0 && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
      return;
    }
  }
  const int64_t n_out = SWIGLU ? p.N / 2 : p.N;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const uint16_t* w = p.w + static_cast<int64_t>(e) * p.N * p.K;
  for (int64_t r0 = 0; r0 < cnt; r0 += 16) {
    float acc = 0.f, acc2 = 0.f;
    const int64_t row = beg + r0 + ty;
    const bool live = r0 + ty < cnt;
    int64_t src = row;
    if (live && p.row_token) {
      src = p.row_token[row];
      if (src < 0 || src >= p.n_x) {
        if (p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
        src = -1;  // a row of zeros
      }
    }
    for (int64_t k0 = 0; k0 < p.K; k0 += 32) {
      for (int c = tx; c < 32; c += 16) {
        const int64_t kk = k0 + c;
        xs[ty][c] = live && src >= 0 && kk < p.K ? bf16_at(p.x, src * p.K + kk) : 0.f;
        ws[ty][c] = n0 + ty < n_out && kk < p.K ? bf16_at(w, (n0 + ty) * p.K + kk) : 0.f;
        if (SWIGLU) us[ty][c] = n0 + ty < n_out && kk < p.K ? bf16_at(w, (n_out + n0 + ty) * p.K + kk) : 0.f;
      }
      __syncthreads();
      for (int c = 0; c < 32; ++c) {
        acc = fmaf(xs[ty][c], ws[tx][c], acc);
        if (SWIGLU) acc2 = fmaf(xs[ty][c], us[tx][c], acc2);
      }
      __syncthreads();
    }
    if (live && n0 + tx < n_out) {
      if (p.low) {
        const int a = p.ids[row];
        if (a >= 0 && a < p.L) {
          const uint16_t* b = p.b + static_cast<int64_t>(a) * p.N * p.R;
          for (int r = 0; r < p.R; ++r) {
            const float v = p.low[row * p.R + r];
            acc = fmaf(v, bf16_at(b, (n0 + tx) * p.R + r), acc);
            if (SWIGLU) acc2 = fmaf(v, bf16_at(b, (n_out + n0 + tx) * p.R + r), acc2);
          }
        }
      }
      if (SWIGLU) acc = silu(acc) * acc2;
      p.out[row * n_out + n0 + tx] = static_cast<uint16_t>(pack_bf16x2(acc, 0.f) & 0xFFFFu);
    }
  }
}

// low[t, r] = scale[a] * A_a[r] . x[t], one warp per (t, r).
__global__ void __launch_bounds__(256)
adapter_shrink_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int32_t* __restrict__ ids,
                      const float* __restrict__ scale, float* __restrict__ low, int64_t T, int64_t K, int R, int L,
                      int32_t* err_flag) {
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  allow_dependent_launch();
  grid_dependency_wait();
  if (job >= T * R) return;
  const int64_t t = job / R;
  const int r = static_cast<int>(job % R);
  const int id = ids[t];
  if (id < 0 || id >= L) {
    if (id >= L && lane == 0 && err_flag) atomicOr(err_flag, MOE_FLAG_BAD_INDEX);
    return;
  }
  const uint16_t* ar = a + (static_cast<int64_t>(id) * R + r) * K;
  float s = 0.f;
  for (int64_t k = lane * 8; k < K; k += 256) {
    float f[8], g[8];
    unpack8(ld_keep16(x + t * K + k), f);
    unpack8(ld_keep16(ar + k), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f[i], g[i], s);
  }
  s = warp_sum(s);
  if (lane == 0) low[t * R + r] = s * scale[id];
}

static cudaError_t launch_linear(const LinearParams& p, int64_t E, int act, cudaStream_t stream) {
  const int64_t n_out = act == MOE_ACT_SWIGLU ? p.N / 2 : p.N;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n_out + 15) / 16), static_cast<unsigned>(E), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return act == MOE_ACT_SWIGLU ? cudaLaunchKernelEx(&cfg, linear_kernel<true>, p)
                               : cudaLaunchKernelEx(&cfg, linear_kernel<false>, p);
}

// Checks common to both products.
static int check_linear(int64_t N, int64_t K, int32_t act) {
  if (N < 1 || K < 1 || (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU)) return MOE_ERR_INVALID_ARG;
  if (N % (act == MOE_ACT_SWIGLU ? 16 : 8) != 0 || K % 8 != 0 || N > MOE_MAX_DIM || K > MOE_MAX_DIM)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

extern "C" int64_t moe_expert_linear_workspace(int64_t n_rows, int64_t E, int64_t N, int64_t K) {
  if (n_rows < 0 || E < 1 || N < 1 || K < 1) return -1;
  return moe::expert_gemm_workspace(n_rows);
}

extern "C" int moe_expert_linear(const void* x_bf16, int64_t n_x, const int32_t* row_token, const void* w_bf16,
                                 const int32_t* offsets, const int32_t* counts, void* out_bf16, int64_t n_rows,
                                 int64_t E, int64_t N, int64_t K, int32_t act, void* workspace,
                                 int64_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
  using namespace moe;
  if (n_x < 0 || n_rows < 0 || E < 1 || workspace_bytes < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(N, K, act);
  if (st != MOE_OK) return st;
  if (E > MOE_MAX_E || n_x > 0x7FFFFFFFll || n_rows > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (!row_token && n_x < n_rows) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if ((n_x > 0 && !x_bf16) || !w_bf16 || !offsets || !counts || !out_bf16) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_expert_linear_workspace(n_rows, E, N, K) || (workspace_bytes > 0 && !workspace))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(out_bf16, 16) || !aligned(workspace, 16) ||
      !aligned(row_token, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(err_flag, 4))
    return MOE_ERR_MISALIGNED;
  const ExpertGemm g{x_bf16, row_token, w_bf16, offsets, counts, out_bf16, n_x, n_rows, E, N, K,
                     act == MOE_ACT_SWIGLU, static_cast<float*>(workspace), err_flag};
  if (launch_expert_gemm(g, stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

extern "C" int64_t moe_adapter_linear_workspace(int64_t T, int64_t N, int64_t K, int32_t R, int32_t L) {
  if (T < 0 || N < 1 || K < 1 || R < 1 || L < 1) return -1;
  return T * R * 4;
}

extern "C" int moe_adapter_linear(const void* x_bf16, const void* w_bf16, const void* adapter_a_bf16,
                                  const void* adapter_b_bf16, const int32_t* adapter_ids,
                                  const float* adapter_scale, void* out_bf16, int64_t T, int64_t N, int64_t K,
                                  int32_t R, int32_t L, int32_t act, void* workspace, int64_t workspace_bytes,
                                  int32_t* err_flag, cudaStream_t stream) {
  using namespace moe;
  if (T < 0 || R < 1 || L < 1 || workspace_bytes < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(N, K, act);
  if (st != MOE_OK) return st;
  if (R % 8 != 0 || R > MOE_MAX_RANK || L > MOE_MAX_ADAPTERS || T > 0x7FFFFFFFll / R) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !w_bf16 || !adapter_a_bf16 || !adapter_b_bf16 || !adapter_ids || !adapter_scale || !out_bf16)
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_adapter_linear_workspace(T, N, K, R, L) || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(adapter_a_bf16, 16) || !aligned(adapter_b_bf16, 16) ||
      !aligned(out_bf16, 16) || !aligned(workspace, 16) || !aligned(adapter_ids, 4) || !aligned(adapter_scale, 4) ||
      !aligned(err_flag, 4))
    return MOE_ERR_MISALIGNED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((T * R + 7) / 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
  cudaError_t e = cudaLaunchKernelEx(&cfg, adapter_shrink_kernel, x, static_cast<const uint16_t*>(adapter_a_bf16),
                                     adapter_ids, adapter_scale, static_cast<float*>(workspace), T, K, R, L, err_flag);
  if (e == cudaSuccess) {
    LinearParams p{};
    p.x = x;
    p.w = static_cast<const uint16_t*>(w_bf16);
    p.out = static_cast<uint16_t*>(out_bf16);
    p.n_x = T;
    p.n_rows = T;
    p.N = N;
    p.K = K;
    p.err_flag = err_flag;
    p.low = static_cast<const float*>(workspace);
    p.b = static_cast<const uint16_t*>(adapter_b_bf16);
    p.ids = adapter_ids;
    p.R = R;
    p.L = L;
    e = launch_linear(p, 1, act, stream);
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return launch_status();
}

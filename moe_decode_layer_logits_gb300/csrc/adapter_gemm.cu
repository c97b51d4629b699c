// moe_adapter_linear: one projection shared by all tokens, with each token's
// low-rank adapter beside it, out[t] = act(W x[t] + s_a B_a (A_a x[t])).
//
// Two forms:
//  - up to kFewTokens tokens (decode): the low-rank products by one warp per
//    (token, rank row); at the same time the shared projection, every tile's
//    K split evenly over all SMs (kParts); then one kernel adds the pieces in
//    order, expands each token's low-rank product against its own B in FP32,
//    applies the activation and rounds once.  Bound by the weights' bytes and,
//    at this size, by three launches' latency.
//  - more tokens: the tokens are sorted by adapter (segments start on multiples
//    of 16 rows), the low-rank products are the expert products of A (kLow),
//    and the shared projection runs in CTA pairs over the sorted rows with the
//    adapters' B as further K blocks of their own columns (kScatter).  A tile of
//    256 rows reads the shared weights once however many adapters it holds.
//    Bound by the tensor cores.
#include "expert_gemm.cuh"
#include "expert_map.h"

namespace moe {

namespace {

constexpr int64_t kFewTokens = kSoloRows;  // one row tile

// low[t, r] = scale[a] * A_a[r] . x[t], one warp per (t, r).
__global__ void __launch_bounds__(256)
adapter_low_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int32_t* __restrict__ ids,
                      const float* __restrict__ scale, float* __restrict__ low, int64_t T, int64_t K, int R, int L,
                      int32_t* err_flag) {
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  // The product that follows starts as soon as this kernel's blocks have
  // waited for the previous one: it reads the same inputs, and this kernel's
  // result only behind its own wait.
  grid_dependency_wait();
  allow_dependent_launch();
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

struct FinishParams {
  const float* partial;
  const float* low;  // [T, R]
  const uint16_t* b;
  const int32_t* ids;
  uint16_t* out;
  int T, N, n_out, R, L, slot_rows;
  int tiles, whole, nkb, G;  // the product's schedule
};

constexpr int kFinishTokens = 8;

// One CTA: 128 weight rows of the product (one of its tiles) and 8 tokens.
template <bool SWIGLU>
__global__ void __launch_bounds__(128) adapter_finish_kernel(const FinishParams p) {
  extern __shared__ float low_s[];  // [kFinishTokens][R]
  __shared__ int id_s[kFinishTokens];
  const int l = threadIdx.x, q = l >> 5, m = blockIdx.x, t0 = blockIdx.y * kFinishTokens;
  allow_dependent_launch();
  grid_dependency_wait();
  const int nt = min(kFinishTokens, p.T - t0);
  for (int i = l; i < kFinishTokens; i += 128) {
    const int a = i < nt ? p.ids[t0 + i] : -1;
    id_s[i] = a < p.L ? a : -1;
  }
  for (int i = l; i < nt * p.R; i += 128) low_s[i] = p.low[static_cast<int64_t>(t0) * p.R + i];
  float v[kFinishTokens];
#pragma unroll
  for (int i = 0; i < kFinishTokens; ++i) v[i] = 0.f;
  auto add = [&](int64_t index) {
    const float* part = p.partial + (index * p.slot_rows + t0) * umma::kBM + l;
#pragma unroll
    for (int i = 0; i < kFinishTokens; ++i)
      if (i < nt) v[i] += part[i * umma::kBM];
  };
  if (m < p.whole) {
    add(parts_index(m, p.G, 0, 0));
  } else {
    const int64_t units = static_cast<int64_t>(p.tiles - p.whole) * p.nkb;
    const int64_t beg = static_cast<int64_t>(m - p.whole) * p.nkb, end = beg + p.nkb;
    auto share = [&](int64_t j) { return units * j / p.G; };
    int j = static_cast<int>(beg * p.G / units);
    while (share(j + 1) <= beg) ++j;
    for (; j < p.G && share(j) < end; ++j)
      if (share(j) < share(j + 1)) add(parts_index(-1, p.G, j, share(j) <= beg ? 0 : 1));
  }
  __syncthreads();
  // this lane's weight row
  const int o = SWIGLU ? m * 64 + q * 16 + (l & 15) : m * 128 + l;
  if (o < p.n_out) {
    const int64_t row = SWIGLU && (l & 16) ? static_cast<int64_t>(p.n_out) + o : o;
    for (int r = 0; r < p.R; r += 8) {
      uint4 b[kFinishTokens];
#pragma unroll
      for (int i = 0; i < kFinishTokens; ++i)
        if (id_s[i] >= 0) b[i] = ld_keep16(p.b + (static_cast<int64_t>(id_s[i]) * p.N + row) * p.R + r);
#pragma unroll
      for (int i = 0; i < kFinishTokens; ++i) {
        if (id_s[i] >= 0) {
          float f[8];
          unpack8(b[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i] = fmaf(low_s[i * p.R + r + e], f[e], v[i]);
        }
      }
    }
  }
  GemmParams g{};
  g.out = p.out;
  g.n_out = p.n_out;
  Piece w{};
  w.r0 = t0;
  w.nr = nt;
  store_cols<SWIGLU, kRows, kFinishTokens>(g, w, m, 0, q, v, 0u);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Places in the workspace.
struct Few {
  int tiles, whole, G, slot_rows;
  size_t low, parts, bytes;
  Few(int64_t T, int64_t N, int R) {
    G = sm_count();
    slot_rows = slot_rows_of(T);
    tiles = static_cast<int>((N + umma::kBM - 1) / umma::kBM);  // gate and up: 64 + 64 rows a tile
    whole = tiles / G * G;
    low = 0;
    parts = up256(static_cast<size_t>(T) * R * 4);
    bytes = parts + (2 * static_cast<size_t>(G) + whole) * slot_rows * umma::kBM * 4;
  }
};

struct Many {
  int64_t n_rows;
  size_t token, seg, counts, low[2], parts, bytes;
  Many(int64_t T, int R, int L) {
    n_rows = moe_expert_rows(T, L + 1, 1, 16);
    token = 0;
    seg = up256(static_cast<size_t>(n_rows) * 4);
    counts = seg + up256((static_cast<size_t>(L) + 2) * 4);
    low[0] = counts + up256((static_cast<size_t>(L) + 1) * 4);
    low[1] = low[0] + up256(static_cast<size_t>(n_rows) * R * 2);
    parts = low[1] + up256(static_cast<size_t>(n_rows) * R * 2);
    bytes = parts + static_cast<size_t>(expert_gemm_workspace(n_rows));
  }
};

template <bool SWIGLU>
cudaError_t few_tokens(const AdapterLinear& g, cudaStream_t stream) {
  const Few f(g.T, g.N, g.R);
  float* low = reinterpret_cast<float*>(g.workspace + f.low);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((g.T * g.R + 7) / 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, adapter_low_kernel, g.x, g.a, g.ids, g.scale, low, g.T, g.K, g.R, g.L,
                                     g.err_flag);
  if (e != cudaSuccess) return e;

  GemmParams p{};
  p.x = g.x;
  p.partial = reinterpret_cast<float*>(g.workspace + f.parts);
  p.err_flag = g.err_flag;
  p.n_rows = g.T;
  p.n_x = static_cast<int>(g.T);
  p.E = 1;
  p.n_out = static_cast<int>(SWIGLU ? g.N / 2 : g.N);
  p.K = static_cast<int>(g.K);
  p.slot_rows = f.slot_rows;
  p.weave = SWIGLU && p.n_out % 16 == 0;
  p.withhold = -1;
  p.wait_late = 1;
  CUtensorMap mx, mw;
  if (!weight_map(&mw, g.w, 1, g.N, g.K, SWIGLU, p.weave) || !row_map_of(&mx, g.x, g.T, g.K, false))
    return cudaErrorInvalidValue;
  e = launch<SWIGLU, false, false, kParts>(mx, mw, mw, p, stream);
  if (e != cudaSuccess) return e;

  const int rows_out = SWIGLU ? 64 : 128;
  const FinishParams fp{p.partial, low, g.b, g.ids, g.out, static_cast<int>(g.T), static_cast<int>(g.N), p.n_out, g.R, g.L,
                        f.slot_rows, (p.n_out + rows_out - 1) / rows_out, f.whole,
                        (p.K + umma::kBK - 1) / umma::kBK, f.G};
  cfg.gridDim = dim3(static_cast<unsigned>(fp.tiles), static_cast<unsigned>((g.T + kFinishTokens - 1) / kFinishTokens), 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(static_cast<size_t>(kFinishTokens) * g.R * 4);
  return cudaLaunchKernelEx(&cfg, adapter_finish_kernel<SWIGLU>, fp);
}

template <bool SWIGLU>
cudaError_t many_tokens(const AdapterLinear& g, cudaStream_t stream) {
  const Many f(g.T, g.R, g.L);
  int32_t* token = reinterpret_cast<int32_t*>(g.workspace + f.token);
  int32_t* seg = reinterpret_cast<int32_t*>(g.workspace + f.seg);
  int32_t* counts = reinterpret_cast<int32_t*>(g.workspace + f.counts);
  // tokens without an adapter are the last segment
  cudaError_t e = launch_expert_map({g.ids, nullptr, token, seg, counts, f.n_rows, g.T, g.L + 1, 1, 16, 1, g.err_flag},
                                    stream);
  if (e != cudaSuccess) return e;

  GemmParams p{};
  p.x = g.x;
  p.row_token = token;
  p.offsets = seg;
  p.counts = counts;
  p.partial = reinterpret_cast<float*>(g.workspace + f.parts);
  p.err_flag = g.err_flag;
  p.n_rows = f.n_rows;
  p.n_x = static_cast<int>(g.T);
  p.E = g.L;
  p.n_out = g.R;
  p.K = static_cast<int>(g.K);
  p.slot_rows = slot_rows_of(f.n_rows);
  p.withhold = -1;
  p.scale = g.scale;
  for (int i = 0; i < 2; ++i) p.low[i] = reinterpret_cast<uint16_t*>(g.workspace + f.low[i]);
  CUtensorMap mx, ma, mw, mb;
  const bool weave = SWIGLU && g.N / 2 % 16 == 0;
  if (!row_map_of(&mx, g.x, g.T, g.K, true) || !weight_map(&ma, g.a, g.L, g.R, g.K, false, false) ||
      !weight_map(&mw, g.w, 1, g.N, g.K, SWIGLU, weave) || !weight_map(&mb, g.b, g.L, g.N, g.R, SWIGLU, weave))
    return cudaErrorInvalidValue;
  e = launch<false, true, false, kLow>(mx, ma, ma, p, stream);
  if (e != cudaSuccess) return e;

  p.offsets = nullptr;
  p.counts = nullptr;
  p.seg = seg;
  p.segs = g.L + 1;
  p.R = g.R;
  p.E = 1;
  p.n_out = static_cast<int>(SWIGLU ? g.N / 2 : g.N);
  p.weave = weave;
  p.out = g.out;
  return launch<SWIGLU, true, true, kScatter>(mx, mw, mb, p, stream);
}

}  // namespace

int64_t adapter_workspace(int64_t T, int64_t N, int64_t K, int R, int L) {
  (void)K;
  return static_cast<int64_t>(T <= kFewTokens ? Few(T, N, R).bytes : Many(T, R, L).bytes);
}

cudaError_t launch_adapter_linear(const AdapterLinear& g, cudaStream_t stream) {
  if (g.T <= kFewTokens) return g.swiglu ? few_tokens<true>(g, stream) : few_tokens<false>(g, stream);
  return g.swiglu ? many_tokens<true>(g, stream) : many_tokens<false>(g, stream);
}

}  // namespace moe

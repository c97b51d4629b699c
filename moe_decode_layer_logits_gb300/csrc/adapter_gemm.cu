// moe_adapter_linear: one projection shared by all tokens, with each token's
// low-rank adapter beside it, out[t] = act(W x[t] + s_a B_a (A_a x[t])).
//
// Two forms:
//  - few tokens (decode): one kernel streams the shared weights, every tile's K
//    split evenly over all SMs (kParts), while further warps of the same CTAs
//    compute the low-rank products, one warp per (token, rank row); a second one
//    adds the pieces in order, expands each token's low-rank product against its
//    own B in FP32, applies the activation and rounds once.  It starts while the
//    first runs and requests the B rows into the L2 meanwhile.  Bound by the
//    weights' bytes and, at this size, by the latency of two launches (K = 6144,
//    N = 4096, R = 16, T = 1: 13.8 us for 7.5 us of bytes; K = 2048, N = 6144,
//    T = 64, 64 adapters: 13.4 for 5.3).
//  - more tokens: the tokens are sorted by adapter (segments start on multiples
//    of 16 rows), the low-rank products are the expert products of A (kLow),
//    and the shared projection runs in CTA pairs over the sorted rows with the
//    adapters' B as further K blocks of their own columns (kScatter).  A tile of
//    256 rows reads the shared weights once however many adapters it holds.
//    Bound by the tensor cores (K = 6144, N = 4096 SwiGLU, R = 64, T = 4096,
//    8 adapters: 181 us, 1170 TFLOP/s; one by one with cold caches the sort
//    takes 10, the low-rank products 22, their join 18, the projection 133).
#include "expert_gemm.cuh"
#include "expert_map.h"

namespace moe {

namespace {

// Few tokens: while the low-rank products (a warp each, and B read by each
// token) and the FP32 partial tiles cost less than the sort and the two further
// products.  64 adapters in use, few / many: K = 2048, N = 6144, T = 64 R = 16
// 13 / 66 us, T = 512 R = 16 38 / 70, T = 256 R = 64 57 / 65, T = 1024 R = 16
// 66 / 79, T = 64 R = 128 76 / 82, T = 16 R = 256 93 / 68; K = 7168, N = 18432,
// R = 16, T = 256 95 / 195, T = 1024 R = 8 305 / 264.  K is not in the rule: at
// K = 7168, N = 18432, T = 512 R = 16 it takes many where few is ahead, 172 / 201.
bool few_form(int64_t T, int64_t N, int R) { return T * N <= 1 << 23 && T * R <= (R <= 128 ? 16384 : 2048); }

struct FinishParams {
  const float* partial;
  const float* low;  // [T, R]
  const uint16_t* b;
  const int32_t* ids;
  uint16_t* out;
  int T, N, n_out, R, L, slot_rows;
  int row_tiles, whole, nkb, G;  // the product's schedule
};

constexpr int kFinishTokens = 8;
constexpr int kFinishPieces = kMaxCtas;  // pieces of one tile: at most one a CTA
constexpr int kFinishBatch = 2;          // pieces loaded at once
constexpr int kFinishPitch = 36;         // words of a row of 64 BF16 columns, and one 16-byte step of padding

// Dynamic shared memory: the tokens' low-rank products, and where the rank asks
// for it four warps' rows of B.
constexpr size_t finish_smem(int R) {
  return static_cast<size_t>(kFinishTokens) * R * 4 + (R > 16 ? 4 * 32 * kFinishPitch * 4 : 0);
}

// One CTA: 128 weight rows of the product and 8 tokens of one of its tiles.
// What follows from the sizes and ids comes before the wait for the product;
// behind it are two rounds of loads (pieces; low-rank products and B).  64
// registers, so that the next product's CTA fits beside the SM's last of these.
template <bool SWIGLU>
__global__ void __launch_bounds__(128, 8) adapter_finish_kernel(const FinishParams p) {
  extern __shared__ float low_s[];  // [kFinishTokens][R]
  __shared__ int id_s[kFinishTokens];
  __shared__ int piece_s[kFinishPieces];
  __shared__ int pieces;
  const int l = threadIdx.x, q = l >> 5, m = blockIdx.x, t0 = blockIdx.y * kFinishTokens;
  allow_dependent_launch();
  const int nt = min(kFinishTokens, p.T - t0);
  if (l < kFinishTokens) {
    const int a = l < nt ? p.ids[t0 + l] : -1;
    id_s[l] = a < p.L ? a : -1;
  }
  // this tile of the list: the row tile that holds t0 (eight tokens lie in one)
  int tt = 0;
  while (tt + 1 < p.row_tiles && tile_begin(p.T, p.row_tiles, tt + 1) <= t0) ++tt;
  const int r0 = tile_begin(p.T, p.row_tiles, tt);
  // its pieces, in the order of K (sizes within 32 bits: fewer tiles than SMs
  // are split, of at most 1024 K blocks each)
  const int tile = m * p.row_tiles + tt;
  if (l < 32) {
    if (tile < p.whole) {
      if (l == 0) {
        piece_s[0] = static_cast<int>(parts_index(tile, p.G, 0, 0));
        pieces = 1;
      }
    } else {
      const unsigned units = (gridDim.x * p.row_tiles - p.whole) * p.nkb, G = p.G;
      const unsigned beg = static_cast<unsigned>(tile - p.whole) * p.nkb, end = beg + p.nkb;
      int n = 0;
      const unsigned from = beg * G / units;
      for (unsigned j0 = from; j0 < G; j0 += 32) {
        const unsigned j = j0 + l, u0 = units * j / G, u1 = units * (j + 1) / G;
        const bool in = j < G && u0 < u1 && u1 > beg && u0 < end;
        const unsigned bal = __ballot_sync(0xFFFFFFFFu, in);
        if (in) piece_s[n + __popc(bal & ((1u << l) - 1u))] = static_cast<int>(parts_index(-1, p.G, j, u0 <= beg ? 0 : 1));
        n += __popc(bal);
        if (units * (j0 + 32) / G >= end) break;
      }
      if (l == 0) pieces = n;
    }
  }
  __syncthreads();
  if (l < 2 * kFinishTokens) {
    const int a = id_s[l >> 1];
    const int per = SWIGLU ? 64 : 128, first = m * per, n = min(per, p.n_out - first);
    if (a >= 0 && (SWIGLU || !(l & 1)))
      prefetch_l2(p.b + (static_cast<int64_t>(a) * p.N + ((l & 1) ? p.n_out : 0) + first) * p.R,
                  static_cast<uint32_t>(n) * p.R * 2);
  }
  const float* part = p.partial + static_cast<int64_t>(t0 - r0) * umma::kBM + l;
  const int64_t step = static_cast<int64_t>(p.slot_rows) * umma::kBM;
  const int o = SWIGLU ? m * 64 + q * 16 + (l & 15) : m * 128 + l;
  const int64_t row = SWIGLU && (l & 16) ? static_cast<int64_t>(p.n_out) + o : o;  // this lane's weight row
  GemmParams g{};
  g.out = p.out;
  g.n_out = p.n_out;
  grid_dependency_wait();
  for (int i = l; i < nt * p.R; i += 128) low_s[i] = p.low[static_cast<int64_t>(t0) * p.R + i];
  float v[kFinishTokens];
#pragma unroll
  for (int i = 0; i < kFinishTokens; ++i) v[i] = 0.f;
  for (int c = 0; c < pieces; c += kFinishBatch) {
    float f[kFinishBatch][kFinishTokens];
#pragma unroll
    for (int j = 0; j < kFinishBatch; ++j)
#pragma unroll
      for (int i = 0; i < kFinishTokens; ++i)
        f[j][i] = c + j < pieces && i < nt ? part[piece_s[c + j] * step + i * umma::kBM] : 0.f;
#pragma unroll
    for (int j = 0; j < kFinishBatch; ++j)
#pragma unroll
      for (int i = 0; i < kFinishTokens; ++i) v[i] += f[j][i];
  }
  __syncthreads();
  if (p.R > 16) {
    // Lanes read whole rows of B together (eight lanes 64 columns of a row) and
    // hand each lane its own row through shared memory; read by the row's lane
    // alone, every load touches 32 lines (29 us at T = 128, R = 64).  The next
    // token's columns are requested before this one's are used; a token with
    // the adapter of the one before finds them in place.
    float* mine = low_s + kFinishTokens * p.R + q * 32 * kFinishPitch;  // this warp's [32 rows][64 columns]
    const int l32 = l & 31, sub = l32 >> 3, chunk = l32 & 7;
    for (int r = 0; r < p.R; r += 64) {
      const int width = min(64, p.R - r);
      uint4 next[8];
      auto request = [&](int id) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int lr = 4 * i + sub;  // row of the warp's 32
          const int oo = SWIGLU ? m * 64 + q * 16 + (lr & 15) : m * 128 + q * 32 + lr;
          const int64_t rr = SWIGLU && (lr & 16) ? static_cast<int64_t>(p.n_out) + oo : oo;
          next[i] = oo < p.n_out && chunk * 8 < width
                        ? ld_keep16(p.b + (static_cast<int64_t>(id) * p.N + rr) * p.R + r + chunk * 8)
                        : make_uint4(0, 0, 0, 0);
        }
      };
      int held = -1, coming = -1;  // adapters whose columns are in shared memory, on their way
      auto following = [&](int i, int id) {  // the next adapter of these tokens that is not `id`
        for (++i; i < nt; ++i)
          if (id_s[i] >= 0 && id_s[i] != id) return id_s[i];
        return -1;
      };
      coming = following(-1, -1);
      if (coming >= 0) request(coming);
      for (int i = 0; i < nt; ++i) {
        const int id = id_s[i];
        if (id < 0) continue;
        if (id != held) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(mine + (4 * k + sub) * kFinishPitch + chunk * 4) = next[k];
          __syncwarp();
          held = id;
          coming = following(i, id);
          if (coming >= 0) request(coming);
        }
        float sum = 0.f;
        for (int c = 0; c < width; c += 8) {
          float f[8];
          unpack8(*reinterpret_cast<const uint4*>(mine + l32 * kFinishPitch + c / 2), f);
          const float* lo = low_s + i * p.R + r + c;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(lo[e], f[e], sum);
        }
#pragma unroll
        for (int k = 0; k < kFinishTokens; ++k)
          if (k == i) v[k] += sum;
      }
      __syncwarp();
    }
  } else if (o < p.n_out) {
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
  Piece w{};
  w.r0 = t0;
  w.nr = nt;
  store_cols<SWIGLU, kRows, kFinishTokens>(g, w, m, 0, q, v, 0u);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Places in the workspace.
struct Few {
  int tiles, row_tiles, whole, G, slot_rows;
  size_t low, parts, bytes;
  Few(int64_t T, int64_t N, int R) {
    G = gemm_ctas();
    slot_rows = slot_rows_of(T);
    row_tiles = static_cast<int>((T + kSoloRows - 1) / kSoloRows);
    tiles = static_cast<int>((N + umma::kBM - 1) / umma::kBM);  // with SwiGLU 64 gate and 64 up rows each
    whole = tiles * row_tiles / G * G;
    low = 0;
    parts = up256(static_cast<size_t>(T) * R * 4);
    bytes = parts + (2 * static_cast<size_t>(G) + whole) * slot_rows * umma::kBM * 4;
  }
};

struct Many {
  int64_t n_rows;
  size_t token, seg, counts, low[kLowParts], parts, bytes;
  Many(int64_t T, int R, int L) {
    n_rows = moe_expert_rows(T, L + 1, 1, 16);
    token = 0;
    seg = up256(static_cast<size_t>(n_rows) * 4);
    counts = seg + up256((static_cast<size_t>(L) + 2) * 4);
    low[0] = counts + up256((static_cast<size_t>(L) + 1) * 4);
    for (int i = 1; i < kLowParts; ++i) low[i] = low[i - 1] + up256(static_cast<size_t>(n_rows) * R * 2);
    parts = low[kLowParts - 1] + up256(static_cast<size_t>(n_rows) * R * 2);
    bytes = parts + static_cast<size_t>(expert_gemm_workspace(n_rows));
  }
};

template <bool SWIGLU>
cudaError_t few_tokens(const AdapterLinear& g, cudaStream_t stream) {
  const Few f(g.T, g.N, g.R);
  float* low = reinterpret_cast<float*>(g.workspace + f.low);
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
  // the last kernel's blocks start beside this one's: with their rows of B they
  // need more of the SM's memory
  p.ring_bytes = g.R > 16 ? kRingBytes - 72 * 1024 : kRingBytes;
  p.weave = SWIGLU && p.n_out % 16 == 0;
  p.withhold = take_withheld_stage();
  p.scale = g.scale;
  p.a = g.a;
  p.ids = g.ids;
  p.low32 = low;
  p.R = g.R;
  p.L = g.L;
  CUtensorMap mx, mw;
  if (!weight_map(&mw, g.w, 1, g.N, g.K, SWIGLU, p.weave) || !row_map_of(&mx, g.x, g.T, g.K))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch<SWIGLU, false, false, kParts>(mx, mw, mw, p, stream);
  if (e != cudaSuccess) return e;

  const FinishParams fp{p.partial, low, g.b, g.ids, g.out, static_cast<int>(g.T), static_cast<int>(g.N), p.n_out, g.R, g.L,
                        f.slot_rows, f.row_tiles, f.whole, (p.K + umma::kBK - 1) / umma::kBK, f.G};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(f.tiles), static_cast<unsigned>((g.T + kFinishTokens - 1) / kFinishTokens), 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = launch_smem(finish_smem(g.R));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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
  p.ring_bytes = kRingBytes;
  p.withhold = take_withheld_stage();
  p.scale = g.scale;
  for (int i = 0; i < kLowParts; ++i) p.low[i] = reinterpret_cast<uint16_t*>(g.workspace + f.low[i]);
  CUtensorMap ma, mw, mb;
  const bool weave = SWIGLU && g.N / 2 % 16 == 0;
  if (!weight_map(&ma, g.a, g.L, g.R, g.K, false, false) || !weight_map(&mw, g.w, 1, g.N, g.K, SWIGLU, weave) ||
      !weight_map(&mb, g.b, g.L, g.N, g.R, SWIGLU, weave))
    return cudaErrorInvalidValue;
  e = launch<false, true, false, kLow>(ma, ma, ma, p, stream);
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
  return launch<SWIGLU, true, true, kScatter>(mw, mw, mb, p, stream);
}

}  // namespace

int64_t adapter_workspace(int64_t T, int64_t N, int64_t K, int R, int L) {
  (void)K;
  return static_cast<int64_t>(few_form(T, N, R) ? Few(T, N, R).bytes : Many(T, R, L).bytes);
}

cudaError_t launch_adapter_linear(const AdapterLinear& g, cudaStream_t stream) {
  if (few_form(g.T, g.N, g.R)) return g.swiglu ? few_tokens<true>(g, stream) : few_tokens<false>(g, stream);
  return g.swiglu ? many_tokens<true>(g, stream) : many_tokens<false>(g, stream);
}

}  // namespace moe

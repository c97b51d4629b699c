// The experts' products on the tensor cores: launches of expert_gemm.cuh.
#include "expert_gemm.cuh"

namespace moe {

namespace {

std::atomic<int> g_withheld{-1};  // take_withheld_stage()

// Pairs from a mean of this many rows an expert, the rows of the call divided
// over all of them.  No device value decides on the host, so those are the rows
// the call has room for: padding and rows of dropped slots count, and a call
// that has much of either runs in pairs with few rows each.  gate_up, E = 256, K = 6144,
// N = 4096, single CTAs / pairs: a mean of 93 rows 1950 / 1951 us, 112 1943 / 1959,
// 128 2188 / 1968; E = 8, a mean of 125 116 / 108.  With room for more rows than
// there are: T = 64 on segments of 128 (2 rows an expert) 1589 / 1643, T = 1024
// with 32 of 256 experts present (33 rows) 252 / 253.  With few tiles: E = 8, a
// mean of 125, N = 256 27 / 32, N = 1024 37 / 36, a mean of 250, N = 2048 83 / 58.
constexpr int64_t kPairMeanRows = 96;

template <bool SWIGLU>
cudaError_t prepare_and_launch(const ExpertGemm& g, cudaStream_t stream) {
  GemmParams p{};
  p.x = static_cast<const uint16_t*>(g.x);
  p.row_token = g.row_token;
  p.offsets = g.offsets;
  p.counts = g.counts;
  p.out = static_cast<uint16_t*>(g.out);
  p.partial = g.partial;
  p.err_flag = g.err_flag;
  p.n_rows = g.n_rows;
  p.n_x = static_cast<int>(g.n_x);
  p.E = static_cast<int>(g.E);
  p.n_out = static_cast<int>(SWIGLU ? g.N / 2 : g.N);
  p.K = static_cast<int>(g.K);
  p.slot_rows = slot_rows_of(g.n_rows);
  p.ring_bytes = kRingBytes;
  p.weave = SWIGLU && p.n_out % 16 == 0;
  p.withhold = take_withheld_stage();

  CUtensorMap mx, mw;
  if (!weight_map(&mw, g.w, g.E, g.N, g.K, SWIGLU, p.weave)) return cudaErrorInvalidValue;
  // pairs copy the rows by their own warps, with a token list or without (four
  // tiled copies a stage beside the weights' were slower by a sixth at T = 8192,
  // E = 256)
  if (g.n_rows / g.E >= kPairMeanRows) return launch<SWIGLU, true, true, kRows>(mw, mw, mw, p, stream);
  if (g.row_token) return launch<SWIGLU, true, false, kRows>(mw, mw, mw, p, stream);
  if (!row_map_of(&mx, g.x, g.n_x, g.K)) return cudaErrorInvalidValue;
  return launch<SWIGLU, false, false, kRows>(mx, mw, mw, p, stream);
}

}  // namespace

int take_withheld_stage() { return g_withheld.exchange(-1); }

int64_t expert_gemm_workspace(int64_t n_rows) {
  return n_rows <= 0 ? 0 : static_cast<int64_t>(gemm_ctas()) * 2 * slot_rows_of(n_rows) * umma::kBM * 4;
}

cudaError_t launch_expert_gemm(const ExpertGemm& g, cudaStream_t stream) {
  return g.swiglu ? prepare_and_launch<true>(g, stream) : prepare_and_launch<false>(g, stream);
}

}  // namespace moe

extern "C" int moe_debug_withhold_expert_stage(int32_t stage) {
  if (stage < -1) return MOE_ERR_INVALID_ARG;
  moe::g_withheld.store(stage);
  return MOE_OK;
}

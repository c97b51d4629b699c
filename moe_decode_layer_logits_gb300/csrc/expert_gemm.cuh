// Products of row segments with their experts' weights on the 5th-generation
// tensor cores: out[r, :] = act(W_e x[src(r)]) for the rows r of segment e
// (device code and launch helpers; expert_gemm.cu and adapter_gemm.cu hold the
// calls).
//
// The weights are the M side (UMMA M = 128 weight rows) and the rows the N
// side with an N of the segment's own size (16 .. 256 in steps of 16), so a
// batch of few rows an expert streams each weight once at the HBM's rate, and
// a large one wastes less than 16 columns a tile.  Persistent CTAs, one per SM:
//  - warp 0 streams 64-wide K blocks of the weights (one TMA copy a stage) and,
//    without a token list, of the rows into a ring of stages of 128-byte
//    swizzled rows;
//  - warp 1 owns the tensor memory, two accumulators of 256 columns, and one
//    lane issues the MMAs;
//  - warps 2..5 read the finished accumulator while the next tile's MMAs run,
//    apply the activation to the FP32 sums and store BF16 once (in pairs, whose
//    tiles have more columns, warps 11..14 too: with four warps the MMAs waited
//    for them a tenth of the time, adapter T = 4096, when its low-rank product
//    had two parts, 182 us against 175);
//  - with a token list the rows are gathered by warps 6..9 with 16-byte
//    asynchronous copies (eight lanes a row of the stage) that arrive on the
//    stage's own barrier as they land, and warp 10 passes that on behind a proxy
//    fence.  (The fence waits for its thread's copies in flight: in the copying
//    warps it left one stage in flight.  A TMA gather of four rows a copy costs
//    the copy engine about 50 cycles whatever its size: 1559 us against 1561 at
//    T = 64, where experts have one or two rows, and 2106 against 1809 at 512.)
// With SwiGLU a tile holds 64 gate and the 64 matching up rows, interleaved by
// 16, so that a gate and its up sit 16 tensor-memory lanes apart, in one warp.
//
// Large segments run in pairs of CTAs (cta_group::2): 256 weight rows and up
// to 256 rows a tile, each CTA loading its 128 weight rows and half of the
// rows, so that every operand byte is read once per pair.
//
// The tile list (segments x row tiles x weight tiles) is made on the device
// from the counts: every CTA scans them.  Single CTAs take row tiles as wide
// as the mean segment asks for (fewer columns leave room for more stages in
// flight).  Whole rounds of the list go round-robin over the CTAs, so that the
// weight tiles of a segment run at the same time and share its rows in the L2;
// the last, partial round is split over all CTAs along K, the pieces are left
// as FP32 partial tiles, and a second small kernel adds them in order (no
// atomics: the same inputs give the same bits).  Pairs take whole tiles.
//
// Measured, SwiGLU, 256 experts of K = 6144, N = 4096, 8 a token, token list:
// even experts unless said otherwise, on two boxes: T = 64 1.56 and 1.60 ms,
// T = 512 1.81 and 1.85 ms (103 to 107% of the copy rate: reads alone are
// faster than a copy), T = 4096 1.97 and 2.02 ms (98 and 96%), T = 8192 uneven
// 2.43 and 2.50 ms (1360 TFLOP/s and 81% of the copy rate in the first), 2.8 ms
// in a second of it (power); with 64 experts, T = 1 70 us (403 MB: 85% of the
// copy rate; the rest is launch, first stages and the join), T = 16384 3.57 and
// 3.78 ms (1850 and 1750 TFLOP/s).  Weights' bytes bound it up to about 150
// rows an expert, the tensor cores where tiles are full; between them both
// matter (a stage turns around in 0.21 us or more whatever its rows, and loads
// that miss the L2 come later than that).
//
// What becomes of the sums is the kernel's Out:
//  - kRows    act, one rounding, row r of the output;
//  - kLow     scaled by the segment, left as three BF16 parts that add up to the
//             FP32 value: the low-rank product of an adapter;
//  - kParts   one segment: every piece left as an FP32 partial tile, for the
//             caller's own last kernel, and the adapters' low-rank products of
//             the rows computed by further warps beside it.  The first stages'
//             weights are requested into the L2 before the wait for the previous
//             kernel (T = 1, K = 6144, N = 4096: 13.4 us; copied into shared
//             memory before it 15.5; two rings of them 14.4);
//  - kScatter rows sorted by adapter, every segment starting on a multiple of
//             16 rows: behind a tile's K blocks come, for each adapter that has
//             rows in the tile, its B against the three parts of its low-rank
//             product, added to that adapter's columns only (so no other token
//             can see it); act, one rounding, the row's token of the output.
#pragma once

#include <atomic>
#include <type_traits>

#include "expert_gemm.h"
#include "host_util.h"
#include "umma.cuh"

namespace moe {

namespace {

constexpr int kMaxStages = 12;
constexpr int kRingBytes = 200 * 1024;
constexpr int kSoloRows = 128;  // most rows of a single CTA's tile (1 << 7)
constexpr int kPairRows = 256;  // rows of a pair's tile (1 << 8)
constexpr int kAccCols = 256;
constexpr int kMaxCtas = 256;   // of a launch
constexpr int kLoaders = 4;     // gathering warps

constexpr int kLowWarps = 8;    // kParts: warps that compute low-rank products
constexpr int kLowParts = 3;    // BF16 parts of a low-rank product: 3 x 8 bits hold FP32's 24

enum Out { kRows, kLow, kParts, kScatter };

// Pairs have a second set of epilogue warps, behind the others.
constexpr int threads_of(bool gather, bool pair, Out out) {
  return 192 + (gather ? 32 * (kLoaders + 1) : 0) + (out == kParts ? 32 * kLowWarps : 0) + (pair ? 128 : 0);
}

struct GemmParams {
  const uint16_t* x;
  const int32_t* row_token;
  const int32_t* offsets;
  const int32_t* counts;
  uint16_t* out;
  float* partial;
  int32_t* err_flag;
  int64_t n_rows;
  int n_x;
  int E, n_out, K;
  int slot_rows;  // rows of a partial tile's slot
  int ring_bytes;
  int weave;      // SwiGLU: one copy brings the whole weight tile (n_out a multiple of 16)
  int withhold;   // test hook: the K block CTA 0 never loads, or -1
  // adapters
  const float* scale;     // kLow, kParts: factor of each
  const uint16_t* a;      // kParts: [L, R, K]
  const int32_t* ids;     // kParts: [n_rows]
  float* low32;           // kParts: [n_rows, R] low-rank products
  int L;
  uint16_t* low[kLowParts];  // kLow, kScatter: [n_rows, R] each
  const int32_t* seg;     // kScatter: [segs + 1] first rows by adapter, then the end
  int segs, R;            // kScatter: the last segment's rows have no adapter
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t landed[kMaxStages];  // gathered rows
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem_base;
  int abort_flag;
  int bn, pieces;
};

__host__ __device__ inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

// The tile list in shared memory: per segment its first row, its rows, and the
// row tiles before it.
struct Tiles {
  int* start;
  int* count;
  int* before;  // E + 1
};

// Rows per tile of single CTAs (a power of two), from the mean rows of the
// segments that have any: the smallest of 32, 64, 128 that leaves room for a
// segment a half larger.
__device__ __forceinline__ int tile_shift(int mean) {
  const int want = mean + (mean + 1) / 2;
  return want <= 32 ? 5 : want <= 64 ? 6 : 7;
}

// Row tiles of the one segment of kScatter: of the few numbers that hold it,
// the one whose rounds over the pairs take the fewest rows.
__device__ __forceinline__ int scatter_tiles(int total, int mt, int G) {
  const int least = (total + kPairRows - 1) / kPairRows;
  int best = least;
  long long cost = -1;
  for (int n = least; n < least + 8 && n > 0; ++n) {
    const long long c = ((static_cast<long long>(n) * mt + G - 1) / G) * round_up((total + n - 1) / n, 16);
    if (cost < 0 || c < cost) {
      cost = c;
      best = n;
    }
  }
  return best;
}

// Row tiles of 2^shift rows that hold `count` rows (up to 2^31 - 1 of them).
__host__ __device__ inline int row_tiles(int count, int shift) {
  return (count >> shift) + ((count & ((1 << shift) - 1)) != 0 ? 1 : 0);
}

// Fills the tile list; every thread of the block calls it.  Afterwards *bn_out
// holds the rows per tile.
template <bool PAIR, Out OUT>
__device__ void list_tiles(const GemmParams& p, Tiles t, int mt, int walkers, int* bn_out, bool report) {
  if (OUT == kParts || OUT == kScatter) {  // one segment, not the caller's
    if (threadIdx.x == 0) {
      const int n = OUT == kScatter ? p.seg[p.segs] : static_cast<int>(p.n_rows);
      const int bn = PAIR ? kPairRows : n <= 32 ? 32 : n <= 64 ? 64 : kSoloRows;
      t.start[0] = 0;
      t.count[0] = n;
      t.before[0] = 0;
      t.before[1] = OUT == kScatter ? scatter_tiles(n, mt, walkers) : (n + bn - 1) / bn;
      *bn_out = bn;
    }
  } else if (threadIdx.x < 32) {
    // lane l takes `per` neighbouring segments, eight loaded at once
    const int lane = threadIdx.x;
    const int per = (p.E + 31) / 32, b = min(p.E, lane * per), e = min(p.E, b + per);
    long long total = 0;
    int active = 0;
    for (int i0 = b; i0 < e; i0 += 8) {
      int beg[8], cnt[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        beg[i] = i0 + i < e ? p.offsets[i0 + i] : 0;
        cnt[i] = i0 + i < e ? p.counts[i0 + i] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i0 + i >= e) break;
        if (beg[i] < 0 || cnt[i] < 0 || static_cast<int64_t>(beg[i]) + cnt[i] > p.n_rows) {  // not inside the rows: skipped
          if (report && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
          beg[i] = 0;
          cnt[i] = 0;
        }
        t.start[i0 + i] = beg[i];
        t.count[i0 + i] = cnt[i];
        total += cnt[i];
        active += cnt[i] > 0 ? 1 : 0;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
      active += __shfl_xor_sync(0xFFFFFFFFu, active, off);
    }
    if (total > p.n_rows) {  // overlapping segments: none is taken
      if (lane == 0 && report && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
      for (int i = b; i < e; ++i) t.count[i] = 0;
      total = 0;
    }
    const int mean = active > 0 ? static_cast<int>((total + active - 1) / active) : 0;
    int shift = PAIR ? 8 : tile_shift(mean);  // rows per tile, as a power of two
    if (OUT == kLow) {
      // narrow weights, so few tiles: the widest rows per tile that still give
      // one for every five CTAs (fewer have too many pieces each to add)
      for (shift = 7; shift > 5; --shift) {
        int tiles = 0;
        for (int i = b; i < e; ++i) tiles += row_tiles(t.count[i], shift);
        if (__reduce_add_sync(0xFFFFFFFFu, tiles) >= static_cast<int>(walkers) / 5) break;
      }
    }
    int mine = 0;
    for (int i = b; i < e; ++i) mine += row_tiles(t.count[i], shift);
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += v;
    }
    int at = upto - mine;
    for (int i = b; i < e; ++i) {
      t.before[i] = at;
      at += row_tiles(t.count[i], shift);
    }
    if (lane == 31) {
      t.before[p.E] = upto;
      *bn_out = 1 << shift;
    }
  }
  __syncthreads();
}

// One piece of work: weight tile m and nr rows from r0 of segment e, K blocks
// [kb0, kb1).  part >= 0: left as an FP32 partial tile at that place.
struct __align__(16) Piece {
  int e, m, r0, nr, kb0, kb1, part, alone;
};

constexpr int kPieces = 256;  // of a walker that are kept in shared memory

// How the tile list is given out to G walkers.  The calls refuse sizes of more
// than 2^31 tiles (an output of that many would not fit any memory), and the
// split round has fewer than kMaxCtas tiles of at most 1024 K blocks, so 32 bits
// hold every number.
struct Schedule {
  unsigned tiles, whole;  // tiles in the list, tiles given out whole
  unsigned rest_units;    // K blocks of the split round
  unsigned mt, nkb, G;    // weight tiles, K blocks, walkers
  __device__ Schedule(const GemmParams& p, const Tiles& t, int weight_tiles, int walkers, bool split)
      : mt(weight_tiles), G(walkers) {
    nkb = (p.K + umma::kBK - 1) / umma::kBK;
    tiles = static_cast<unsigned>(t.before[p.E]) * mt;
    whole = split ? tiles / G * G : tiles;
    rest_units = (tiles - whole) * nkb;
  }
  // Start of walker b's share of the split round.
  __device__ unsigned share(unsigned b) const { return rest_units * b / G; }
  // Whole tiles of walker b (b, b + G, ...), and all its pieces: its share is
  // no longer than a tile and so lies in at most two.
  __device__ unsigned whole_of(unsigned b) const { return whole > b ? (whole - b + G - 1) / G : 0; }
  __device__ int pieces(unsigned b) const {
    unsigned n = whole_of(b);
    if (rest_units > 0) {
      const unsigned u = share(b), left = share(b + 1) - u;
      if (left > 0) n += u % nkb + left > nkb ? 2 : 1;
    }
    return static_cast<int>(n);
  }
};

// Rows of row tile tt of ntt of a segment: nearly the same number of sixteens
// each.
__host__ __device__ inline int tile_begin(int cnt, int ntt, int tt) {
  const int sixteens = cnt / 16 + (cnt % 16 != 0 ? 1 : 0), each = sixteens / ntt, more = sixteens % ntt;
  const int at = (each * tt + (tt < more ? tt : more));
  return at >= sixteens ? cnt : at * 16;
}

// Tile `tile` of the list.
__device__ __forceinline__ void locate(const Tiles& t, int E, unsigned mt, unsigned tile, Piece& w) {
  const int at = static_cast<int>(tile / mt);
  int lo = 0, hi = E;  // before[lo] <= at < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.before[mid] <= at) lo = mid;
    else hi = mid;
  }
  const unsigned ntt = t.before[lo + 1] - t.before[lo], local = tile - t.before[lo] * mt;
  w.e = lo;
  w.alone = ntt == 1;
  w.r0 = t.start[lo];
  w.nr = t.count[lo];
  w.m = static_cast<int>(local);
  if (ntt > 1) {
    w.m = static_cast<int>(local / ntt);
    const int tt = static_cast<int>(local % ntt);
    const int a = tile_begin(w.nr, static_cast<int>(ntt), tt), b = tile_begin(w.nr, static_cast<int>(ntt), tt + 1);
    w.r0 += a;
    w.nr = b - a;
  }
}

// Places of the partial tiles.  A walker has at most one piece of the split
// round that starts a tile (kb0 == 0), and one that does not; kParts leaves its
// whole tiles too, behind them.
__host__ __device__ inline int64_t parts_index(int64_t whole_tile, int G, int cta, int kb0) {
  return whole_tile >= 0 ? 2 * static_cast<int64_t>(G) + whole_tile : 2 * static_cast<int64_t>(cta) + (kb0 == 0 ? 1 : 0);
}

// Piece i of a walker.
__device__ __forceinline__ Piece make_piece(const Schedule& s, const Tiles& t, int E, unsigned who, unsigned i, bool parts) {
  Piece w;
  const unsigned whole = s.whole_of(who);
  if (i < whole) {
    const unsigned tile = who + i * s.G;
    locate(t, E, s.mt, tile, w);
    w.kb0 = 0;
    w.kb1 = static_cast<int>(s.nkb);
    w.part = parts ? static_cast<int>(parts_index(tile, s.G, 0, 0)) : -1;
    return w;
  }
  unsigned u = s.share(who);
  const unsigned end = s.share(who + 1);
  unsigned nth = u / s.nkb;
  if (i > whole) u = ++nth * s.nkb;
  locate(t, E, s.mt, s.whole + nth, w);
  w.kb0 = static_cast<int>(u - nth * s.nkb);
  w.kb1 = static_cast<int>(min(s.nkb, w.kb0 + (end - u)));
  w.part = !parts && w.kb0 == 0 && w.kb1 == static_cast<int>(s.nkb) ? -1 : static_cast<int>(parts_index(-1, s.G, who, w.kb0));
  return w;
}

// The same for the warps of a walker with more than kPieces pieces, as one copy
// of the code.
__device__ __noinline__ void make_far_piece(const Schedule& s, const Tiles& t, int E, unsigned who, unsigned i, bool parts,
                                            Piece* w) {
  *w = make_piece(s, t, E, who, i, parts);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// Whether row r's token names a row of x.
__device__ __forceinline__ bool token_ok(const GemmParams& p, int r) {
  const int s = p.row_token[r];
  return s >= 0 && s < p.n_x;
}

// Rows c .. c + 31 of the tile whose token names no row (one bit a row): they
// are stored as zeros.
__device__ __forceinline__ unsigned bad_rows(const GemmParams& p, const Piece& w, int c) {
  const int r = c + (threadIdx.x & 31);
  return p.row_token ? __ballot_sync(0xFFFFFFFFu, r < w.nr && !token_ok(p, w.r0 + r)) : 0u;
}

// Stores NC columns (rows r0 + c ..) of one weight tile; v[i] is this lane's
// weight row for row i.  Neighbouring lanes swap halves of two rows so that
// each store covers a whole row piece of the warp.  m: the 128-row weight tile.
// aux: kRows the bad rows' bits, kScatter the token of row c + lane, kLow the
// factor's bits.
template <bool SWIGLU, Out OUT, int NC>
__device__ __forceinline__ void store_cols(const GemmParams& p, const Piece& w, int m, int c, int q,
                                           const float (&v)[NC], unsigned aux) {
  const int lane = threadIdx.x & 31;
  const int left = w.nr - c;
  // lanes of a row: 0..15 hold gates and 16..31 their ups (after the swap the
  // lower half finishes row i, the upper half row i + 1); without SwiGLU even
  // and odd lanes share out the two rows
  const bool second = SWIGLU ? lane >= 16 : lane & 1;
  const int o = SWIGLU ? m * 64 + q * 16 + (lane & 15) : m * 128 + q * 32 + (lane & ~1);
#pragma unroll
  for (int i = 0; i < NC; i += 2) {
    const float other = __shfl_xor_sync(0xFFFFFFFFu, second ? v[i] : v[i + 1], SWIGLU ? 16 : 1);
    const float a = second ? other : v[i], b = second ? v[i + 1] : other;
    const int r = second ? i + 1 : i;
    int64_t row = static_cast<int64_t>(w.r0) + c + r;
    bool live = r < left && o < p.n_out;
    if (OUT == kScatter) {
      const int t0 = __shfl_sync(0xFFFFFFFFu, static_cast<int>(aux), i);
      const int t1 = __shfl_sync(0xFFFFFFFFu, static_cast<int>(aux), i + 1);
      row = second ? t1 : t0;
      live = live && row >= 0;
    }
    if (OUT == kLow) {
      const float f = __uint_as_float(aux), x = f * a, y = f * b;
      // each part is what BF16 holds of what the ones before leave, which FP32
      // holds exactly; an infinite value leaves nothing, and a finite one beyond
      // BF16's largest starts with that
      float rx = x, ry = y;
#pragma unroll
      for (int part = 0; part < kLowParts; ++part) {
        uint32_t u = pack_bf16x2(rx, ry);
        if (part == 0) {
          if (isfinite(x) && isinf(bf16lo(u))) --u;
          if (isfinite(y) && isinf(bf16hi(u))) u -= 0x10000u;
        }
        if (live) *reinterpret_cast<uint32_t*>(p.low[part] + row * p.n_out + o) = u;
        rx = isfinite(x) ? rx - bf16lo(u) : 0.f;
        ry = isfinite(y) ? ry - bf16hi(u) : 0.f;
      }
    } else {
      const bool bad = OUT == kRows && ((aux >> r) & 1u);
      if (SWIGLU) {
        const float y = bad ? 0.f : silu_mul(a, b);
        if (live) p.out[row * p.n_out + o] = static_cast<uint16_t>(pack_bf16x2(y, 0.f));
      } else if (live) {
        *reinterpret_cast<uint32_t*>(p.out + row * p.n_out + o) = bad ? 0u : pack_bf16x2(a, b);
      }
    }
  }
}

// store_cols' aux for rows c .. of a tile.
template <Out OUT>
__device__ __forceinline__ unsigned store_aux(const GemmParams& p, const Piece& w, int c) {
  if (OUT == kLow) return __float_as_uint(p.scale[w.e]);
  if (OUT == kScatter) {
    const int r = c + (threadIdx.x & 31);
    return static_cast<unsigned>(r < w.nr ? p.row_token[w.r0 + r] : -1);
  }
  return bad_rows(p, w, c);
}

// The adapters of a tile, in the order in which all warps walk them: columns
// [c0, c0 + n) of the tile against adapter a.
struct Adapters {
  int a, r0, r1, c0, n;
  __device__ Adapters(const GemmParams& p, const int* seg, const Piece& w) : r0(w.r0), r1(w.r0 + w.nr) {
    int lo = 0, hi = p.segs;  // the last segment that starts at or before r0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seg[mid] <= r0) lo = mid;
      else hi = mid;
    }
    a = lo - 1;
  }
  __device__ bool get(const GemmParams& p, const int* seg) {
    while (++a < p.segs - 1) {
      const int b = max(seg[a], r0), e = min(seg[a + 1], r1);
      if (seg[a] >= r1) return false;
      if (e > b) {
        c0 = b - r0;
        n = e - b;
        return true;
      }
    }
    return false;
  }
};

template <bool SWIGLU, bool GATHER, bool PAIR, Out OUT>
// (the bounds: registers that leave room for the next kernel's blocks beside it)
__global__ void __launch_bounds__(OUT == kParts ? 768 : 512, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_b, const __grid_constant__ GemmParams p) {
  static_assert(!PAIR || GATHER, "pairs copy their rows by warps 6 to 9");
  static_assert(OUT != kScatter || PAIR, "sorted rows run in pairs");
  using namespace umma;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers sb;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Piece* piece_s = reinterpret_cast<Piece*>(ring + p.ring_bytes);
  int* list = reinterpret_cast<int*>(piece_s + kPieces);
  const Tiles t{list, list + p.E, list + 2 * p.E};
  int* seg = list + 3 * p.E + 1;  // kScatter: the adapters' first rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int who = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  volatile int* abort_v = &sb.abort_flag;

  if (threadIdx.x < kMaxStages) {
    // a stage is full when its copies have landed and, where other warps gather
    // the rows, they have been reported (by each CTA of a pair)
    mbar_init(&sb.full[threadIdx.x], 1 + (GATHER ? (PAIR ? 2 : 1) : 0));
    mbar_init(&sb.landed[threadIdx.x], 32 * kLoaders);
    mbar_init(&sb.empty[threadIdx.x], 1);
    mbar_init_fence();
  } else if (threadIdx.x < kMaxStages + 2) {
    mbar_init(&sb.acc_full[threadIdx.x - kMaxStages], 1);
    mbar_init(&sb.acc_empty[threadIdx.x - kMaxStages], PAIR ? 16 : 4);
    mbar_init_fence();
  } else if (threadIdx.x == kMaxStages + 2) {
    mbar_init(&sb.drained, 1);
    sb.abort_flag = 0;
    mbar_init_fence();
  } else if (threadIdx.x == kMaxStages + 3) {
    prefetch_map(&tmap_w);
    if (!GATHER) prefetch_map(&tmap_x);
  }
  if (warp == 1) tmem_alloc<PAIR>(&sb.tmem_base, 2 * kAccCols);
  if (OUT != kParts) {
    // the trigger comes behind the wait, so that what is launched next finds
    // this kernel's own inputs ready
    grid_dependency_wait();
    allow_dependent_launch();
  }
  const int rows_out = (SWIGLU ? 64 : 128) * (PAIR ? 2 : 1), mt = (p.n_out + rows_out - 1) / rows_out;
  const int walkers = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);
  if (OUT == kScatter)
    for (int i = threadIdx.x; i <= p.segs; i += blockDim.x) seg[i] = p.seg[i];
  list_tiles<PAIR, OUT>(p, t, mt, walkers, &sb.bn, blockIdx.x == 0);  // kParts: reads no global memory
  const int depth = OUT == kScatter ? (p.R + kBK - 1) / kBK : 0;  // K blocks of an adapter's B
  // this walker's pieces, one a thread
  const Schedule s(p, t, mt, walkers, !PAIR);
  {
    const int n = s.pieces(who);
    if (threadIdx.x == 0) sb.pieces = n;
    for (int i = threadIdx.x; i < min(n, kPieces); i += blockDim.x) piece_s[i] = make_piece(s, t, p.E, who, i, OUT == kParts);
  }
  fence_before_sync();
  __syncthreads();
  if (PAIR) {  // the peer's barriers are ready before anything signals them
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  fence_after_sync();
  const uint32_t tmem = sb.tmem_base;
  // a stage: 128 weight rows, then this CTA's rows (a pair's CTA holds half of the tile's)
  const int stage_bytes = (kBM + (PAIR ? kPairRows / 2 : sb.bn)) * kRowBytes;
  const int nstages = min(kMaxStages, p.ring_bytes / stage_bytes);
  // A ring position and its parity; no division in the stage loops (with one
  // each, every warp's turn took a tenth of the HBM's rate at T = 64).
  struct Stage {
    int st, ph;
  };
  auto advance = [&](Stage& x) {
    if (++x.st == nstages) {
      x.st = 0;
      x.ph ^= 1;
    }
  };
  const int pieces = sb.pieces;
  // all warps walk the pieces in the same order
  auto next = [&](int& at, Piece& w) {
    if (at >= pieces) return false;
    if (at < kPieces) {
      w = piece_s[at];
    } else {
      Piece made;  // (a reference to w itself would keep it out of the registers)
      make_far_piece(s, t, p.E, who, at, OUT == kParts, &made);
      w = made;
    }
    ++at;
    return true;
  };
  // barriers that the first CTA of a pair keeps for both
  const uint32_t full0 = PAIR ? cluster_addr(&sb.full[0], 0) : smem_addr(&sb.full[0]);
  const uint32_t acc_empty0 = PAIR ? cluster_addr(&sb.acc_empty[0], 0) : smem_addr(&sb.acc_empty[0]);

  if (warp == 0) {
    // -------------------------------------------------------------- loads
    if (elect_one()) {  // one lane walks and copies
      const uint64_t once = l2_evict_first_policy(), keep = l2_evict_normal_policy();
      const int withheld = who == 0 ? p.withhold : -1;
      auto load_weights = [&](const CUtensorMap* map, uint32_t dst, int kb, int m, int e, uint32_t bar, uint64_t pol) {
        if (!SWIGLU) {
          tma_load_5d<PAIR>(dst, map, kb * kBK, m * 128, 0, 0, e, bar, pol);
        } else if (p.weave) {
          tma_load_5d<PAIR>(dst, map, kb * kBK, 0, 0, m * 4, e, bar, pol);
        } else {  // 16 gate rows and their 16 up rows at a time
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tma_load_5d<PAIR>(dst + i * 32 * kRowBytes, map, kb * kBK, m * 64 + i * 16, 0, 0, e, bar, pol);
        }
      };
      // bytes of a stage's copies, in both CTAs of a pair
      auto stage_copies = [&](const Piece& w) {
        return static_cast<uint32_t>((PAIR ? 2 : 1) * kBM + (GATHER ? 0 : round_up(w.nr, 32))) * kRowBytes;
      };
      int at = 0;
      Piece w;
      int n = 0;  // stages so far
      Stage x{0, 0};
      if (OUT == kParts) {
        // a ring of weights into the L2 before the wait (not into shared memory: a
        // kernel still running may write them)
        int ahead = 0, early = 0;
        while (early < nstages && next(ahead, w)) {
          for (int kb = w.kb0; kb < w.kb1 && early < nstages; ++kb, ++early) {
            if (!SWIGLU) {
              tma_prefetch_5d(&tmap_w, kb * kBK, w.m * 128, 0, 0, w.e);
            } else if (p.weave) {
              tma_prefetch_5d(&tmap_w, kb * kBK, 0, 0, w.m * 4, w.e);
            } else {
              for (int i = 0; i < 4; ++i) tma_prefetch_5d(&tmap_w, kb * kBK, w.m * 64 + i * 16, 0, 0, w.e);
            }
          }
        }
        grid_dependency_wait();
        // behind the wait, so that what is launched next finds the inputs ready
        allow_dependent_launch();
      }
      bool stop = false;
      // the next stage may be written: its last MMAs are done
      auto freed = [&]() { return n < nstages || wait(&sb.empty[x.st], x.ph ^ 1, abort_v); };
      while (!stop && next(at, w)) {
        const int boxes = GATHER ? 0 : (w.nr + 31) >> 5;
        const uint32_t bytes = stage_copies(w);
        const int m = PAIR ? w.m * 2 + rank : w.m;
        const uint64_t pol = w.alone ? once : keep;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++n, advance(x)) {
          if (!freed()) {
            stop = true;
            break;
          }
          if (n == withheld) continue;  // neither armed nor loaded: the MMA warp's wait runs out
          const uint32_t a = smem_addr(ring) + static_cast<uint32_t>(x.st * stage_bytes);
          const uint32_t b = a + kBM * kRowBytes, bar = full0 + x.st * 8;
          if (rank == 0) mbar_arrive_expect_tx(&sb.full[x.st], bytes);
          load_weights(&tmap_w, a, kb, m, w.e, bar, pol);
          for (int i = 0; i < boxes; ++i) tma_load_2d(b + i * 32 * kRowBytes, &tmap_x, kb * kBK, w.r0 + i * 32, bar);
        }
        if (OUT == kScatter && !stop) {
          Adapters ad(p, seg, w);
          while (!stop && ad.get(p, seg)) {
            for (int i = 0; i < kLowParts * depth; ++i, ++n, advance(x)) {
              if (!freed()) {
                stop = true;
                break;
              }
              if (rank == 0) mbar_arrive_expect_tx(&sb.full[x.st], 2 * kBM * kRowBytes);
              load_weights(&tmap_b, smem_addr(ring) + static_cast<uint32_t>(x.st * stage_bytes), i / kLowParts, m, ad.a,
                           full0 + x.st * 8, keep);
            }
          }
        }
      }
      // drain: no copy may land after this CTA exits (a pair's copies are counted
      // by its first CTA, and neither leaves before the other)
      if (rank == 0) {
        const int from = n > nstages ? n - nstages : 0;
        Stage y{from % nstages, (from / nstages) & 1};
        for (int i = from; i < n; ++i, advance(y))
          if (i != withheld) wait(&sb.full[y.st], y.ph, abort_v, true);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (rank == 0 && elect_one()) {
      // before the first bounded wait, whose probes are for this kernel's own
      // loads: those begin behind the previous kernel, which may run long
      if (OUT == kParts) grid_dependency_wait();
      int at = 0;
      Piece w;
      const uint32_t a0 = desc_low(smem_addr(ring)), step = static_cast<uint32_t>(stage_bytes) >> 4;
      Stage x{0, 0};
      int seq = 0;
      bool stop = false;
      while (!stop && next(at, w)) {
        const int acc = seq & 1, use = seq >> 1;
        if (use > 0 && !wait(&sb.acc_empty[acc], (use - 1) & 1, abort_v)) break;
        fence_after_sync();
        const uint32_t d = tmem + acc * kAccCols;
        const uint32_t idesc = idesc_bf16(PAIR ? 2 * kBM : kBM, round_up(w.nr, 16));
        for (int kb = w.kb0; kb < w.kb1; ++kb, advance(x)) {
          const int st = x.st;
          if (!wait(&sb.full[st], x.ph, abort_v)) {
            stop = true;
            break;
          }
          fence_after_sync();
          const uint32_t a = a0 + static_cast<uint32_t>(st) * step, b = a + (kBM * kRowBytes >> 4);
          mma_bf16<PAIR>(d, a, b, idesc, kb != w.kb0);
#pragma unroll
          for (int kk = 1; kk < kBK / 16; ++kk) mma_bf16<PAIR>(d, a + kk * 2, b + kk * 2, idesc, true);
          mma_commit<PAIR>(&sb.empty[st]);
        }
        if (OUT == kScatter && !stop) {
          Adapters ad(p, seg, w);
          while (!stop && ad.get(p, seg)) {
            const uint32_t sub = idesc_bf16(2 * kBM, ad.n);
            for (int i = 0; i < kLowParts * depth; ++i, advance(x)) {
              const int st = x.st;
              if (!wait(&sb.full[st], x.ph, abort_v)) {
                stop = true;
                break;
              }
              fence_after_sync();
              const uint32_t a = a0 + static_cast<uint32_t>(st) * step, b = a + (kBM * kRowBytes >> 4);
              const int ks = (min(kBK, p.R - i / kLowParts * kBK) + 15) >> 4;
              for (int kk = 0; kk < ks; ++kk) mma_bf16<PAIR>(d + ad.c0, a + kk * 2, b + kk * 2, sub, true);
              mma_commit<PAIR>(&sb.empty[st]);
            }
          }
        }
        if (stop) break;  // (a peer's epilogue must not take half a sum for a whole one)
        mma_commit<PAIR>(&sb.acc_full[acc]);
        ++seq;
      }
      mma_commit<PAIR>(&sb.drained);  // also after an abort: fires once the issued MMAs are done
    }
    __syncwarp();
  } else if (warp < 6 || (PAIR && warp > 6 + kLoaders)) {
    // ----------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp's quarter of the tensor-memory lanes
    if (OUT == kParts) grid_dependency_wait();
    int at = 0;
    Piece w;
    int seq = 0;
    bool dead = false;  // a wait ran out: this and all later pieces are left as NaN
    while (next(at, w)) {
      const int acc = seq & 1, use = seq >> 1;
      ++seq;
      if (!dead) {
        const bool ok = wait(&sb.acc_full[acc], use & 1, abort_v) && !*abort_v;
        dead = !__all_sync(0xFFFFFFFFu, ok);
      }
      fence_after_sync();
      const uint32_t d = tmem + acc * kAccCols + (static_cast<uint32_t>(q * 32) << 16);
      float* part = p.partial + static_cast<int64_t>(w.part) * p.slot_rows * kBM + q * 32 + lane;
#pragma unroll 1
      for (int c = PAIR && warp >= 6 ? 32 : 0; c < w.nr; c += PAIR ? 64 : 32) {  // two sets of warps take turns
        uint32_t raw[32];
        if (!dead) {
          tmem_ld32(d + static_cast<uint32_t>(c), raw);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) raw[i] = 0x7FC00000u;
        }
        if (OUT == kParts || w.part >= 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < w.nr) part[(c + i) * kBM] = __uint_as_float(raw[i]);
        } else {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
          store_cols<SWIGLU, OUT, 32>(p, w, PAIR ? w.m * 2 + rank : w.m, c, q, v, store_aux<OUT>(p, w, c));
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0 && !dead) {
        if (PAIR) arrive_cluster(acc_empty0 + acc * 8);
        else mbar_arrive(&sb.acc_empty[acc]);
      }
    }
  } else if (OUT == kParts) {
    // -------------------------------------------------- low-rank products
    // low32[t, r] = scale[a] * A_a[r] . x[t]: a warp takes one rank row of a
    // token, or two neighbouring ones where there are several rounds of them
    grid_dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kLowWarps + warp - 6;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kLowWarps;
    auto products = [&](auto rows) {
      constexpr int RB = decltype(rows)::value;
      const int per = p.R / RB;
      for (int64_t job = first; job < p.n_rows * per; job += warps) {
        const int64_t row = job / per;
        const int r = static_cast<int>(job - row * per) * RB, id = p.ids[row];
        if (id < 0 || id >= p.L) {
          if (id >= p.L && lane == 0 && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
          continue;
        }
        const uint16_t* ar = p.a + (static_cast<int64_t>(id) * p.R + r) * p.K;
        const uint16_t* xr = p.x + row * p.K;
        float sum[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) sum[i] = 0.f;
#pragma unroll(RB == 1 ? 6 : 4)
        for (int k = lane * 8; k < p.K; k += 256) {
          float f[8], g[8];
          unpack8(ld_keep16(xr + k), f);
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            unpack8(ld_stream16(ar + static_cast<int64_t>(i) * p.K + k), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[i] = fmaf(f[e], g[e], sum[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          sum[i] = warp_sum(sum[i]);
          if (lane == 0) p.low32[row * p.R + r + i] = sum[i] * p.scale[id];
        }
      }
    };
    if (p.n_rows * p.R > 2 * warps) products(std::integral_constant<int, 2>{});
    else products(std::integral_constant<int, 1>{});
  } else if (GATHER && warp < 6 + kLoaders) {
    // ------------------------------------------------------------- gather
    // Warp j takes rows 16 i + 4 j .. + 3 of this CTA's rows, eight lanes a
    // row, 16 bytes a lane, at their place in the 128-byte swizzle.
    const int j = warp - 6, sub = lane >> 3, chunk = lane & 7;
    const uint32_t place = static_cast<uint32_t>((kBM + 4 * j + sub) * kRowBytes + ((chunk ^ ((4 * j + sub) & 7)) << 4));
    int at = 0;
    Piece w;
    int n = 0;
    Stage x{0, 0};
    bool stop = false;
    while (!stop && next(at, w)) {
      const int mine = PAIR ? round_up(w.nr, 16) / 2 : w.nr;  // rows in this CTA, at most 128
      // Rows without a token of their own are not copied: what the stage holds
      // there reaches only columns that are not stored, or stored as zeros.
      const uint16_t* src[8];
      unsigned live = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 16 * i + 4 * j + sub, rr = rank * mine + r;
        int tok = -1;
        if (r < mine && rr < w.nr) {
          tok = p.row_token ? p.row_token[w.r0 + rr] : w.r0 + rr;
          if (tok < 0 || tok >= p.n_x) {
            tok = -1;
            if (OUT != kScatter && p.err_flag) atomicOr(p.err_flag, MOE_FLAG_BAD_INDEX);
          }
        }
        live |= tok >= 0 ? 1u << i : 0u;
        src[i] = p.x + static_cast<int64_t>(max(tok, 0)) * p.K + chunk * 8 + w.kb0 * kBK;
      }
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n, advance(x)) {
        const int st = x.st;
        if (n >= nstages && !wait(&sb.empty[st], x.ph ^ 1, abort_v)) {
          stop = true;
          break;
        }
        const uint32_t b = smem_addr(ring) + static_cast<uint32_t>(st * stage_bytes) + place;
        const bool inside = kb * kBK + chunk * 8 < p.K;  // zeros behind the end of K
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((live >> i) & 1u) copy16_async(b + i * 16 * kRowBytes, src[i], inside);
          src[i] += kBK;
        }
        copy_arrive(&sb.landed[st]);
      }
      if (OUT == kScatter && !stop) {
        Adapters ad(p, seg, w);
        while (!stop && ad.get(p, seg)) {
          const int half = ad.n / 2;
          const int64_t first = w.r0 + ad.c0 + rank * half;
          for (int i = 0; i < kLowParts * depth; ++i, ++n, advance(x)) {
            const int st = x.st;
            if (n >= nstages && !wait(&sb.empty[st], x.ph ^ 1, abort_v)) {
              stop = true;
              break;
            }
            const uint32_t b = smem_addr(ring) + static_cast<uint32_t>(st * stage_bytes + kBM * kRowBytes);
            const int col = i / kLowParts * kBK + chunk * 8;
            const uint16_t* low = p.low[i % kLowParts];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
              const int r = 16 * h + 4 * j + sub;
              if (r < half) {
                const bool live = col < p.R;
                copy16_async(b + r * kRowBytes + ((chunk ^ (r & 7)) << 4), low + (live ? (first + r) * p.R + col : 0),
                             live);
              }
            }
            copy_arrive(&sb.landed[st]);
          }
        }
      }
    }
    copy_drain();
  } else if (GATHER) {
    // -------------------------------------------------- gathered rows are in
    if (lane == 0) {
      int at = 0;
      Piece w;
      Stage x{0, 0};
      bool stop = false;
      while (!stop && next(at, w)) {
        int stages = w.kb1 - w.kb0;
        if (OUT == kScatter) {
          Adapters ad(p, seg, w);
          while (ad.get(p, seg)) stages += kLowParts * depth;
        }
        for (int i = 0; i < stages; ++i, advance(x)) {
          const int st = x.st;
          if (!wait(&sb.landed[st], x.ph, abort_v)) {
            stop = true;
            break;
          }
          proxy_fence();
          if (PAIR) arrive_cluster(full0 + st * 8);
          else mbar_arrive(&sb.full[st]);
        }
      }
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 32) wait(&sb.drained, 0, abort_v, true);  // no MMA is in flight any more
  __syncwarp();
  if (PAIR) {  // the peer's copies and arrivals are over too
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  if (threadIdx.x == 0 && p.err_flag && *abort_v) atomicOr(p.err_flag, MOE_FLAG_TIMEOUT);
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc<PAIR>(tmem, 2 * kAccCols);
  }
}

// Adds the partial tiles of the split round.  CTA (b, y) takes the tile at the
// end of share b if that end lies inside it and no earlier share ends there,
// and of its rows those with row / 16 % gridDim.y == y.  What follows from the
// segments comes before the wait for the products, which start this kernel
// behind their own wait.  (At most 85 registers: it fits on an SM beside them.)
constexpr int kJoinBatch = 2;  // pieces loaded at once

template <bool SWIGLU, Out OUT>
__global__ void __launch_bounds__(128, 6) expert_join_kernel(const GemmParams p, int G) {
  extern __shared__ int join_list[];
  __shared__ int bn, pieces;
  __shared__ int piece_s[kMaxCtas];
  const Tiles t{join_list, join_list + p.E, join_list + 2 * p.E};
  allow_dependent_launch();
  const int rows_out = SWIGLU ? 64 : 128, mt = (p.n_out + rows_out - 1) / rows_out;
  list_tiles<false, OUT>(p, t, mt, G, &bn, false);
  const Schedule s(p, t, mt, G, true);
  const int b = blockIdx.x, l = threadIdx.x, q = l >> 5;
  const unsigned end = s.share(b + 1), tile0 = end / s.nkb * s.nkb;
  // the share ends between two tiles, or an earlier share ends in this tile
  const bool none = end == tile0 || end >= s.rest_units || s.share(b) > tile0;
  Piece w{};
  if (!none) {
    locate(t, p.E, s.mt, s.whole + end / s.nkb, w);
    if (l < 32) {  // the tile's pieces in the order of K: this share's start of it, then the next shares'
      int n = 1;
      if (l == 0) piece_s[0] = static_cast<int>(parts_index(-1, G, b, 0));
      for (int j0 = b + 1; j0 < G; j0 += 32) {
        const int j = j0 + l;
        const unsigned u0 = s.share(min(j, G)), u1 = s.share(min(j + 1, G));
        const bool in = u0 < u1 && u0 < tile0 + s.nkb;
        const unsigned bal = __ballot_sync(0xFFFFFFFFu, in);
        if (in) piece_s[n + __popc(bal & ((1u << l) - 1u))] = static_cast<int>(parts_index(-1, G, j, 1));
        n += __popc(bal);
        if (s.share(min(j0 + 32, G)) >= tile0 + s.nkb) break;
      }
      if (l == 0) pieces = n;
    }
  }
  __syncthreads();
  const int64_t step = static_cast<int64_t>(p.slot_rows) * umma::kBM;
  // The first pass, before the wait, has no rows: it only brings the
  // instructions into the caches (3.4 us behind the wait without it).
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) grid_dependency_wait();
    if (none) continue;
    const int nr = pass == 1 ? w.nr : 0;
    for (int c = blockIdx.y * 16; c < max(nr, static_cast<int>(blockIdx.y) * 16 + 1); c += gridDim.y * 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
      const float* part = p.partial + static_cast<int64_t>(c) * umma::kBM + l;
      for (int j = 0; j < pieces; j += kJoinBatch) {
        float f[kJoinBatch][16];
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            f[k][i] = j + k < pieces && c + i < nr ? part[piece_s[j + k] * step + i * umma::kBM] : 0.f;
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += f[k][i];
      }
      Piece rows = w;
      rows.nr = nr;
      store_cols<SWIGLU, OUT, 16>(p, rows, w.m, c, q, v, store_aux<OUT>(p, rows, c));
    }
  }
}

// ---------------------------------------------------------------- host side

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load();
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      fn.store(f);
    }
  }
  return f;
}

// Row-major BF16 tensor of `rank` dimensions (innermost first), 128-byte swizzle.
inline bool make_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a launch: one per SM.
inline int gemm_ctas() { return sm_count() < kMaxCtas ? sm_count() : kMaxCtas; }

// Dynamic shared memory: the ring, the walker's pieces, the tile list, the adapters' first rows.
inline size_t gemm_smem(int64_t E, int segs, int ring) {
  return 1024 + static_cast<size_t>(ring) + kPieces * sizeof(Piece) + static_cast<size_t>(3 * E + 1 + segs + 1) * sizeof(int);
}

// Opt the kernel into its dynamic shared memory, once per device.
template <bool SWIGLU, bool GATHER, bool PAIR, Out OUT>
cudaError_t opt_in(int dev) {
  static std::atomic<bool> done[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(expert_gemm_kernel<SWIGLU, GATHER, PAIR, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(gemm_smem(OUT == kScatter ? 1 : MOE_MAX_E, OUT == kScatter ? MOE_MAX_ADAPTERS + 1 : 0, kRingBytes)));
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  return cudaSuccess;
}

template <bool SWIGLU, bool GATHER, bool PAIR, Out OUT>
cudaError_t launch(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mb, const GemmParams& p,
                   cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = opt_in<SWIGLU, GATHER, PAIR, OUT>(dev);
  if (e != cudaSuccess) return e;
  const int G = PAIR ? gemm_ctas() / 2 * 2 : gemm_ctas();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(G), 1, 1);
  cfg.blockDim = dim3(threads_of(GATHER, PAIR, OUT), 1, 1);
  cfg.dynamicSmemBytes = launch_smem(gemm_smem(p.E, p.segs, p.ring_bytes));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (PAIR) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<SWIGLU, GATHER, PAIR, OUT>, mx, mw, mb, p);
  if constexpr (!PAIR && (OUT == kRows || OUT == kLow)) {
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(G - 1), static_cast<unsigned>((p.slot_rows + 15) / 16), 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = launch_smem(static_cast<size_t>(3 * p.E + 1) * sizeof(int));
    e = cudaLaunchKernelEx(&cfg, expert_join_kernel<SWIGLU, OUT>, p, G);
  }
  return e;
}

// Rows of a partial tile's slot.
inline int slot_rows_of(int64_t n_rows) {
  return static_cast<int>(n_rows < kSoloRows ? round_up(static_cast<int>(n_rows), 16) : kSoloRows);
}

// Weights as (K, N, 1, 1, E); SwiGLU: (K, n_out, gate / up, 1, E), or (K, 16,
// gate / up, n_out / 16, E) where n_out divides (`weave`), so that one box is a
// whole interleaved tile.
inline bool weight_map(CUtensorMap* map, const void* w, int64_t E, int64_t N, int64_t K, bool swiglu, bool weave) {
  const cuuint64_t row = static_cast<cuuint64_t>(K) * 2, n = static_cast<cuuint64_t>(swiglu ? N / 2 : N);
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(K), weave ? 16 : n, swiglu ? 2u : 1u, weave ? n / 16 : 1,
                              static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[4] = {row, row * n, row * 16, row * static_cast<cuuint64_t>(N)};
  const cuuint32_t box[5] = {umma::kBK, swiglu ? 16u : 128u, swiglu ? 2u : 1u, weave ? 4u : 1u, 1u};
  return make_map(map, w, 5, dims, strides, box);
}

// Rows of x in boxes of 32.
inline bool row_map_of(CUtensorMap* map, const void* x, int64_t n_x, int64_t K) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(n_x)}, row = static_cast<cuuint64_t>(K) * 2;
  const cuuint32_t box[2] = {umma::kBK, 32};
  return make_map(map, x, 2, dims, &row, box);
}

}  // namespace
}  // namespace moe

// Rows sorted by expert and back (moe_permute, moe_unpermute) and their gradients
// (ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference",
// Abstract: every selected expert of a step executes; grouping a step's pairs by expert
// is what a grouped product needs).
//
// With R the T*k x T matrix that holds w[p] at (pair_pos[p], p / k), the four calls are
// rows = R x, out = R^T rows, and the transposes of these in their gradients, which add
// the scalar products that are the weights' gradients.  So one kernel either spreads a
// token's row over its k sorted rows or gathers them, with or without the scalar
// products.  It goes by token, whose row is read (written) once.
//
// Bound by HBM where there are many tokens.  T = 4096, d = 2048, k = 8 in bf16: 26.5 us for
// 151 MB (5.7 TB/s; a plain copy of 1 GiB runs at 5.0), back 26.7 us, the gradient of the
// way back with the products 54 us for 286 MB (5.3 TB/s).  16 tokens take 3.4 us and one
// 2.1: a launch and two dependent loads, the positions and then the rows.
#include "rows.hpp"

namespace moe {

struct PermuteDev {
  const void* token_in;   // spread: the token rows (x, dout); gather with products: x
  int64_t token_in_stride;
  const void* sorted_in;  // gather: the sorted rows (rows, drows); spread with products: rows
  int64_t sorted_in_stride;
  void* out;              // spread: the sorted rows; gather: the token rows
  int64_t out_stride;
  int64_t num_rows;
  int T, d, k;
  float* dweights;        // products only
};

// How the threads of a workgroup share tokens: a token has 1 << lt lanes of a wavefront
// (short rows) or `waves` whole ones, and each lane `rounds` pieces of its row.
struct TokenSplit {
  int lt, waves, tokens, threads, rounds;
};

// Elements that belong to the piece before are in its sum: here both factors of their
// products become zero (an infinite one times zero would be NaN).  The masks are vector
// registers.  As conditions of the sums they would take scalar ones, which the sorted rows'
// addresses fill (permute gradient, d = 4864, k = 12, T = 768 in fp32: 54.9 in place of 50.4 us;
// T = 16384, d = 200, k = 8 in fp16: 18.7 in place of 15.2).
__device__ __forceinline__ uint32_t own_mask(const Piece& p, int i) {
  uint32_t m = i < p.skip ? 0u : ~0u;
  asm("" : "+v"(m));
  return m;
}
__device__ __forceinline__ float masked(float v, uint32_t mask) { return __uint_as_float(__float_as_uint(v) & mask); }

// Rows of more than 256 elements.  A wavefront handles 64 pieces of 8 elements of one
// token with at most KM pairs: its positions and weights come through scalar loads, the
// rows' addresses are scalar, and the loads of KB rows go out before the first use.  Up to
// four pairs fit the scalar registers in every form, eight without products.  With more of
// them some wait in lanes of vector registers (25 to 41 for eight pairs with products, two
// bytes gathered excepted; for sixteen 14 to 48, floats gathered 116, and 130 to 226 with
// products).  Pairs that were dropped read some row that is there (`sorted_in` always has
// one) and are masked, so that no load sits under a branch.
// kStream: the sorted rows start on 16-byte boundaries.  Then they are read, each once, by
// non-temporal loads (unpermute at T = 4096, d = 2048, k = 8: 29.0 to 26.8 us); off them
// two lanes share a cache line, which would be fetched twice (odd gradient 4.8 to 5.5 us).
template <typename S, bool kSpread, bool kProducts, int KM, int KB, bool kStream>
__global__ __launch_bounds__(1024) void k_rows(PermuteDev a, const int32_t* __restrict__ pair_pos,
                                               const float* __restrict__ weights, TokenSplit p) {
  __shared__ float part_sums[kProducts ? 16 : 1][KM];
  // Spread alone, rows of two bytes off 16-byte boundaries go through the L2, which puts the
  // lines together that they end in (T = 4096, d = 1111, k = 8 23.2 to 15.9 us).  With
  // products, whose loads the L2 has to hold, it does not pay (29.8 to 37.5 us).
  constexpr bool kPast = kProducts || kStream || sizeof(S) == 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int part = wave % p.waves, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * p.tokens + wave / p.waves;
  const bool live = t < a.T;
  if (!live && !kProducts) return;
  const int64_t tc = live ? t : a.T - 1;
  int64_t pos[KM];
  float w[KM], dot[KM];
  uint32_t kept[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    const int64_t at = tc * a.k + (j < a.k ? j : a.k - 1);
    pos[j] = pair_pos[at];
    w[j] = weights ? weights[at] : 1.f;
    dot[j] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    kept[j] = live && j < a.k && pos[j] >= 0 && pos[j] < a.num_rows ? ~0u : 0u;
    pos[j] = kept[j] ? pos[j] : 0;
    w[j] = kept[j] ? w[j] : 0.f;  // (times a masked row: an infinite weight would make NaN of it)
  }
  for (int it = 0; it < p.rounds; ++it) {
    const Piece c = piece_of((part * 64 + lane + it * p.waves * 64) * kPiece, a.d);
    Raw<S> mine;
    if (kSpread || kProducts)
      mine = load_raw<false>(row_ptr<S, false>(a.token_in, tc, a.token_in_stride), c, a.d);
    float v[kPiece], own[kPiece], r[kPiece], acc[kPiece];
    uint32_t mask[kPiece];
    if (kSpread || kProducts) unpack<S>(mine, v);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      acc[i] = 0.f;
      if (kProducts) own[i] = masked(v[i], mask[i] = own_mask(c, i));
    }
#pragma unroll
    for (int j0 = 0; j0 < KM; j0 += KB) {
      if (j0 >= a.k) continue;
      Raw<S> row[KB];
      if (!kSpread || kProducts) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
          row[b] = load_raw<false, kStream>(row_ptr<S, false>(a.sorted_in, pos[j0 + b], a.sorted_in_stride), c, a.d);
      }
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const int j = j0 + b;
        if (!kSpread || kProducts) {
          unpack<S>(masked<S>(row[b], kept[j]), r);
#pragma unroll
          for (int i = 0; i < kPiece; ++i) {
            if (!kSpread) acc[i] = fmaf(w[j], r[i], acc[i]);
            if (kProducts) dot[j] = fmaf(own[i], masked(r[i], mask[i]), dot[j]);
          }
        }
        if (kSpread && kept[j]) {
          S* dst = row_ptr<S, false>(a.out, pos[j], a.out_stride);
          if (weights) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) acc[i] = w[j] * v[i];
            store_piece<false, kPast>(dst, c, a.d, acc);
          } else {
            store_raw<false, kPast>(dst, c, a.d, mine);
          }
        }
      }
      if (KB < KM) __builtin_amdgcn_sched_barrier(0);
    }
    if (!kSpread && live) store_piece<false>(row_ptr<S, false>(a.out, tc, a.out_stride), c, a.d, acc);
  }
  if constexpr (kProducts) {
    // over the lanes, then over the token's wavefronts in order
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      dot[j] = lane_sum(dot[j], 6);
      if (lane == 0) part_sums[wave][j] = kept[j] ? dot[j] : 0.f;
    }
    __syncthreads();
    if (!live || part != 0 || lane >= a.k) return;
    float s = 0.f;
    for (int i = 0; i < p.waves; ++i) s += part_sums[wave + i][lane];
    a.dweights[t * a.k + lane] = s;
  }
}

// Rows of at most 256 elements: 1 << lt lanes per token, several tokens per wavefront (a
// whole wavefront per token would leave half of its lanes idle or more).  Spread alone they go
// through the L2: most such rows end inside lines (T = 16384, k = 8 in bf16: d = 250 25.3 to
// 14.9 us, 81 11.5 to 9.4, but 128 7.8 to 9.0; in fp32 250 71 to 41).
template <typename S, bool kSpread, bool kProducts>
__global__ __launch_bounds__(256) void k_rows_short(PermuteDev a, const int32_t* __restrict__ pair_pos,
                                                    const float* __restrict__ weights, TokenSplit p) {
  const int lane = threadIdx.x & ((1 << p.lt) - 1);
  const int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> p.lt;
  if (t >= a.T) return;  // (a token's lanes return together: the sums below stay within them)
  const Piece c = piece_of(lane * kPiece, a.d);
  Raw<S> mine{};
  if (kSpread || kProducts) mine = load_raw<true>(row_ptr<S, true>(a.token_in, t, a.token_in_stride), c, a.d);
  float v[kPiece], own[kPiece], r[kPiece], acc[kPiece];
  uint32_t mask[kPiece];
  unpack<S>(mine, v);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    acc[i] = 0.f;
    own[i] = masked(v[i], mask[i] = own_mask(c, i));
  }
  for (int j = 0; j < a.k; ++j) {
    const int64_t at = t * a.k + j, pos = pair_pos[at];
    const bool kept = pos >= 0 && pos < a.num_rows;
    const float w = !kept ? 0.f : weights ? weights[at] : 1.f;
    float dot = 0.f;
    if (!kSpread || kProducts) {
      Raw<S> row = load_raw<true>(row_ptr<S, true>(a.sorted_in, kept ? pos : 0, a.sorted_in_stride), c, a.d);
      unpack<S>(masked<S>(row, kept ? ~0u : 0u), r);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        if (!kSpread) acc[i] = fmaf(w, r[i], acc[i]);
        if (kProducts) dot = fmaf(own[i], masked(r[i], mask[i]), dot);
      }
    }
    if (kSpread && kept) {
      S* dst = row_ptr<S, true>(a.out, pos, a.out_stride);
      if (weights) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) r[i] = w * v[i];
        store_piece<true, kProducts>(dst, c, a.d, r);
      } else {
        store_raw<true, kProducts>(dst, c, a.d, mine);
      }
    }
    if (kProducts) {
      dot = lane_sum(dot, p.lt);
      if (lane == 0) a.dweights[at] = kept ? dot : 0.f;
    }
  }
  if (!kSpread) store_piece<true>(row_ptr<S, true>(a.out, t, a.out_stride), c, a.d, acc);
}

// At most 16 wavefronts share a token, four where they hold much of it: the sums of the
// products, or more than eight sorted rows.  Larger workgroups leave registers of a CU over
// (d = 4288, T = 1011, bf16, nine wavefronts against three with three pieces per lane:
// gradient of the way back k = 8 34.3 and 30.3 us, of permute 21.1 and 17.0, unpermute k = 12
// 24.6 and 22.6; the others lose by it, permute k = 8 19.3 and 20.9, unpermute 14.7 and 15.0).
// Tokens of which every CU has one at most keep all: their time is that of one token's rounds
// (permute gradient, d = 4864, k = 12 in fp32: T = 128 17.4 and 26.3 us, T = 768 57.7 and 50.6;
// nothing between the two was timed).
static TokenSplit token_split(int T, int d, bool heavy) {
  TokenSplit p;
  const int pieces = (int)ceil_div(d, kPiece);
  p.lt = 0;
  while (p.lt < 6 && (1 << p.lt) < pieces) ++p.lt;
  const int64_t full = ceil_div(pieces, 64);
  p.rounds = (int)ceil_div(full, heavy && T > 256 ? 4 : 16);
  p.waves = (int)ceil_div(full, p.rounds);
  p.tokens = p.lt < 6 ? 256 >> p.lt : std::max(1, 4 / p.waves);
  p.threads = p.lt < 6 ? 256 : p.tokens * p.waves * 64;
  return p;
}

static int launch_rows(const char* name, int timing_id, bool spread, int dtype, PermuteDev a, const int32_t* pair_pos,
                       const float* weights, hipStream_t s) {
  const TokenSplit p = token_split(a.T, a.d, a.dweights || (!spread && a.k > 8));
  const dim3 grid((unsigned)ceil_div(a.T, p.tokens));
  if (a.num_rows == 0) {  // every pair is dropped: what they read is masked, any row will do
    a.sorted_in = spread ? a.token_in : a.out;
    a.sorted_in_stride = 0;
  }
  timing_begin(timing_id, s);
  with_dtype(dtype, [&](auto v) {
    using S = decltype(v);
    auto go = [&](auto spread_c, auto products_c, auto stream_c) {
      constexpr bool kSpread = decltype(spread_c)::value, kProducts = decltype(products_c)::value;
      constexpr bool kStream = decltype(stream_c)::value;
      auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(p.threads), 0, s, a, pair_pos, weights, p); };
      if (p.lt < 6)
        launch(k_rows_short<S, kSpread, kProducts>);
      else if (a.k <= 2)
        launch(k_rows<S, kSpread, kProducts, 2, 2, kStream>);
      else if (a.k <= 4)
        launch(k_rows<S, kSpread, kProducts, 4, 4, kStream>);
      else if (a.k <= 8)
        launch(k_rows<S, kSpread, kProducts, 8, 8, kStream>);
      else
        // (all rows of a token at once where the registers hold them: unpermute, T = 4096,
        // d = 2048, k = 12 in bf16 41.6 to 37.5 us)
        launch(k_rows<S, kSpread, kProducts, 16, sizeof(S) == 2 && !kSpread && !kProducts ? 16 : 8, kStream>);
    };
    const std::true_type yes;
    const std::false_type no;
    const bool products = a.dweights != nullptr;
    const void* sorted = spread && !products ? a.out : a.sorted_in;
    const int64_t sorted_stride = spread && !products ? a.out_stride : a.sorted_in_stride;
    const bool stream = ((uintptr_t)sorted | (uintptr_t)(sorted_stride * (int64_t)sizeof(S))) % 16 == 0;
    if (spread && !products)
      stream ? go(yes, no, yes) : go(yes, no, no);
    else if (spread)
      stream ? go(yes, yes, yes) : go(yes, yes, no);
    else if (a.dweights)
      stream ? go(no, yes, yes) : go(no, yes, no);
    else
      stream ? go(no, no, yes) : go(no, no, no);
  });
  timing_end(timing_id, s);
  return check_launch(name);
}

// one of the row tensors of a call
struct RowArg {
  const char* name;
  const void* ptr;
  int64_t stride;
  bool output, wanted;
};

static int check_rows(const char* fn, int dtype, int T, int d, int k, int64_t num_rows, const void* pair_pos,
                      const void* weights, const void* dweights, const RowArg (&rows)[4]) {
  MOE_CHECK_ARG(dtype >= MOE_BF16 && dtype <= MOE_FP32, MOE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  MOE_CHECK_ARG(T >= 0 && d > 0 && k > 0 && num_rows >= 0, MOE_ERR_INVALID_ARG,
                "%s: bad sizes T=%d d=%d k=%d num_rows=%lld", fn, T, d, k, (long long)num_rows);
  MOE_CHECK_ARG(k <= MOE_MAX_TOPK && (int64_t)T * k <= (1 << 24) && d <= (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: unsupported k=%d T*k=%lld d=%d (k <= 16, T*k <= 2^24, d <= 2^24)", fn, k, (long long)T * k, d);
  MOE_CHECK_ARG((int64_t)T * d <= kMaxRowElements, MOE_ERR_UNSUPPORTED_SHAPE, "%s: unsupported T*d=%lld (<= 2^34)",
                fn, (long long)T * d);
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(pair_pos && ((uintptr_t)pair_pos % 4) == 0 && ((uintptr_t)weights % 4) == 0 &&
                    ((uintptr_t)dweights % 4) == 0,
                MOE_ERR_INVALID_ARG, "%s: pair_pos is NULL, or pair_pos, weights or dweights misaligned", fn);
  const int64_t size = dtype_bytes(dtype);
  for (const RowArg& r : rows) {
    if (!r.wanted) continue;
    MOE_CHECK_ARG(r.ptr && ((uintptr_t)r.ptr % size) == 0, MOE_ERR_INVALID_ARG, "%s: %s is NULL or misaligned", fn,
                  r.name);
    MOE_CHECK_ARG(r.stride >= (r.output ? d : 0), MOE_ERR_INVALID_ARG, "%s: stride %lld of %s below %d", fn,
                  (long long)r.stride, r.name, r.output ? d : 0);
  }
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_permute(const void* x, int64_t x_stride, int dtype, int T, int d, int k, const int32_t* pair_pos,
                           const float* weights, void* rows, int64_t rows_stride, int64_t num_rows, void* stream) {
  clear_error();
  const RowArg args[4] = {{"x", x, x_stride, false, true}, {"rows", rows, rows_stride, true, num_rows > 0}, {}, {}};
  const int rc = check_rows("moe_permute", dtype, T, d, k, num_rows, pair_pos, weights, nullptr, args);
  if (rc || T == 0) return rc;
  const PermuteDev a{x, x_stride, nullptr, 0, rows, rows_stride, num_rows, T, d, k, nullptr};
  return launch_rows("moe_permute", K_PERMUTE, true, dtype, a, pair_pos, weights, (hipStream_t)stream);
}

extern "C" int moe_unpermute(const void* rows, int64_t rows_stride, int64_t num_rows, int dtype, int T, int d, int k,
                             const int32_t* pair_pos, const float* weights, void* out, int64_t out_stride,
                             void* stream) {
  clear_error();
  const RowArg args[4] = {{"rows", rows, rows_stride, false, num_rows > 0}, {"out", out, out_stride, true, true}, {}, {}};
  const int rc = check_rows("moe_unpermute", dtype, T, d, k, num_rows, pair_pos, weights, nullptr, args);
  if (rc || T == 0) return rc;
  const PermuteDev a{nullptr, 0, rows, rows_stride, out, out_stride, num_rows, T, d, k, nullptr};
  return launch_rows("moe_unpermute", K_UNPERMUTE, false, dtype, a, pair_pos, weights, (hipStream_t)stream);
}

extern "C" int moe_permute_backward(const void* drows, int64_t drows_stride, int64_t num_rows, const void* x,
                                    int64_t x_stride, int dtype, int T, int d, int k, const int32_t* pair_pos,
                                    const float* weights, void* dx, int64_t dx_stride, float* dweights, void* stream) {
  clear_error();
  const RowArg args[4] = {{"drows", drows, drows_stride, false, num_rows > 0},
                          {"x", x, x_stride, false, dweights != nullptr},
                          {"dx", dx, dx_stride, true, true},
                          {}};
  const int rc = check_rows("moe_permute_backward", dtype, T, d, k, num_rows, pair_pos, weights, dweights, args);
  if (rc || T == 0) return rc;
  const PermuteDev a{x, x_stride, drows, drows_stride, dx, dx_stride, num_rows, T, d, k, dweights};
  return launch_rows("moe_permute_backward", K_UNPERMUTE, false, dtype, a, pair_pos, weights, (hipStream_t)stream);
}

extern "C" int moe_unpermute_backward(const void* dout, int64_t dout_stride, const void* rows, int64_t rows_stride,
                                      int dtype, int T, int d, int k, const int32_t* pair_pos, const float* weights,
                                      void* drows, int64_t drows_stride, int64_t num_rows, float* dweights,
                                      void* stream) {
  clear_error();
  const RowArg args[4] = {{"dout", dout, dout_stride, false, true},
                          {"rows", rows, rows_stride, false, dweights != nullptr && num_rows > 0},
                          {"drows", drows, drows_stride, true, num_rows > 0},
                          {}};
  const int rc = check_rows("moe_unpermute_backward", dtype, T, d, k, num_rows, pair_pos, weights, dweights, args);
  if (rc || T == 0) return rc;
  const PermuteDev a{dout, dout_stride, rows, rows_stride, drows, drows_stride, num_rows, T, d, k, dweights};
  return launch_rows("moe_unpermute_backward", K_PERMUTE, true, dtype, a, pair_pos, weights, (hipStream_t)stream);
}

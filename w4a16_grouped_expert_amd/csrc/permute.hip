// Rows sorted by expert and back (moe_permute, moe_unpermute) and their gradients
// (ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference",
// Abstract: every selected expert of a step executes; grouping a step's pairs by expert
// is what a grouped product needs).
//
// With R the T*k x T matrix that holds w[p] at (pair_pos[p], p / k), the four calls are
// rows = R x, out = R^T rows, and the transposes of these in their gradients, which add
// the scalar products that are the weights' gradients.  So there are two kernels, one
// that spreads a token's row over its k sorted rows and one that gathers them, each with
// or without the scalar products.  Both go by token: its row is read (written) once.
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
  const int32_t* pair_pos;
  const float* weights;   // or null
  float* dweights;        // products only
};

// One group of 1 << lt lanes per token (lt <= 6), 64 >> lt tokens per wavefront.
template <typename S, bool kProducts, bool kTiny>
__global__ __launch_bounds__(256) void k_spread(PermuteDev a, int lt) {
  const int lane = threadIdx.x & ((1 << lt) - 1);
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lt;
  const bool live = t < a.T;
  const int64_t tc = live ? t : a.T - 1;
  const S* src = static_cast<const S*>(a.token_in) + tc * a.token_in_stride;
  float dot[MOE_MAX_TOPK];
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOPK; ++j) dot[j] = 0.f;
  for (int c = lane * kPiece; c < a.d; c += kPiece << lt) {
    const Piece n = piece_of(c, a.d);
    Raw<S> raw = load_raw<kTiny>(src, n, a.d);
    mask_piece(raw, n);
    float v[kPiece];
    unpack<S>(raw, v);
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      const int64_t pos = j < a.k ? a.pair_pos[tc * a.k + j] : -1;
      if (!live || pos < 0 || pos >= a.num_rows) continue;
      if constexpr (kProducts) {
        float r[kPiece];
        load_piece<kTiny>(static_cast<const S*>(a.sorted_in) + pos * a.sorted_in_stride, n, a.d, r);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) dot[j] = fmaf(v[i], r[i], dot[j]);
      }
      S* dst = static_cast<S*>(a.out) + pos * a.out_stride;
      if (a.weights) {
        const float w = a.weights[tc * a.k + j];
        float o[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) o[i] = w * v[i];
        store_piece<kTiny>(dst, n, a.d, o);
      } else {
        store_raw<kTiny>(dst, n, a.d, raw);
      }
    }
  }
  if constexpr (kProducts) {
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      const float s = lane_sum(dot[j], lt);
      if (live && lane == 0 && j < a.k) a.dweights[t * a.k + j] = s;
    }
  }
}

template <typename S, bool kProducts, bool kTiny>
__global__ __launch_bounds__(256) void k_gather(PermuteDev a, int lt) {
  const int lane = threadIdx.x & ((1 << lt) - 1);
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lt;
  const bool live = t < a.T;
  const int64_t tc = live ? t : a.T - 1;
  float dot[MOE_MAX_TOPK];
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOPK; ++j) dot[j] = 0.f;
  for (int c = lane * kPiece; c < a.d; c += kPiece << lt) {
    const Piece n = piece_of(c, a.d);
    float v[kPiece], acc[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) acc[i] = 0.f;
    if constexpr (kProducts)
      load_piece<kTiny>(static_cast<const S*>(a.token_in) + tc * a.token_in_stride, n, a.d, v);
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      const int64_t pos = j < a.k ? a.pair_pos[tc * a.k + j] : -1;
      if (!live || pos < 0 || pos >= a.num_rows) continue;
      const float w = a.weights ? a.weights[tc * a.k + j] : 1.f;
      float r[kPiece];
      load_piece<kTiny>(static_cast<const S*>(a.sorted_in) + pos * a.sorted_in_stride, n, a.d, r);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        acc[i] = fmaf(w, r[i], acc[i]);
        if constexpr (kProducts) dot[j] = fmaf(v[i], r[i], dot[j]);
      }
    }
    if (live) store_piece<kTiny>(static_cast<S*>(a.out) + t * a.out_stride, n, a.d, acc);
  }
  if constexpr (kProducts) {
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      const float s = lane_sum(dot[j], lt);
      if (live && lane == 0 && j < a.k) a.dweights[t * a.k + j] = s;
    }
  }
}

// lanes per token (log2): as many as have a piece of the row, at most a wavefront
static int token_lanes_log2(int d) {
  int lt = 0;
  while (lt < 6 && (kPiece << lt) < d) ++lt;
  return lt;
}

static int launch_rows(const char* name, int timing_id, bool spread, int dtype, const PermuteDev& a, hipStream_t s) {
  const int lt = token_lanes_log2(a.d);
  const dim3 grid((unsigned)ceil_div((int64_t)a.T << lt, 256));
  const bool products = a.dweights != nullptr;
  timing_begin(timing_id, s);
  with_dtype(dtype, [&](auto v) {
    using S = decltype(v);
    auto go = [&](auto prod, auto tiny) {
      constexpr bool kP = decltype(prod)::value, kT = decltype(tiny)::value;
      if (spread)
        hipLaunchKernelGGL((k_spread<S, kP, kT>), grid, dim3(256), 0, s, a, lt);
      else
        hipLaunchKernelGGL((k_gather<S, kP, kT>), grid, dim3(256), 0, s, a, lt);
    };
    const bool tiny = a.d < kPiece;
    if (products)
      tiny ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else
      tiny ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
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
  const PermuteDev a{x, x_stride, nullptr, 0, rows, rows_stride, num_rows, T, d, k, pair_pos, weights, nullptr};
  return launch_rows("moe_permute", K_PERMUTE, true, dtype, a, (hipStream_t)stream);
}

extern "C" int moe_unpermute(const void* rows, int64_t rows_stride, int64_t num_rows, int dtype, int T, int d, int k,
                             const int32_t* pair_pos, const float* weights, void* out, int64_t out_stride,
                             void* stream) {
  clear_error();
  const RowArg args[4] = {{"rows", rows, rows_stride, false, num_rows > 0}, {"out", out, out_stride, true, true}, {}, {}};
  const int rc = check_rows("moe_unpermute", dtype, T, d, k, num_rows, pair_pos, weights, nullptr, args);
  if (rc || T == 0) return rc;
  const PermuteDev a{nullptr, 0, rows, rows_stride, out, out_stride, num_rows, T, d, k, pair_pos, weights, nullptr};
  return launch_rows("moe_unpermute", K_UNPERMUTE, false, dtype, a, (hipStream_t)stream);
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
  const PermuteDev a{x, x_stride, drows, drows_stride, dx, dx_stride, num_rows, T, d, k, pair_pos, weights, dweights};
  return launch_rows("moe_permute_backward", K_UNPERMUTE, false, dtype, a, (hipStream_t)stream);
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
  const PermuteDev a{dout,     dout_stride, rows, rows_stride, drows,   drows_stride, num_rows,
                     T,        d,           k,    pair_pos,    weights, dweights};
  return launch_rows("moe_unpermute_backward", K_PERMUTE, true, dtype, a, (hipStream_t)stream);
}

// Dropout of row tensors with the residual's addition, for training the blocks whose layers
// around the routed experts stay in BF16 (ExactMoE, page "Every Expert Counts: ExactMoE for
// Memory-Efficient W4A16 Inference", Abstract; of training and dropout the page says nothing).
//
//   out[r][c] = residual[r][c] + (keep(r, c) ? x[r][c] / (1 - p) : 0)
//
// keep comes from philox.hpp.  The gradient is the same call on dout without a residual.
//
// A lane holds one piece of a row: the eight columns of one generator call in 16-bit types
// (16 bytes), four floats.  Bound by memory: two or three tensors cross it once (T = 16384,
// d = 2048, bf16 with the residual: 35.7 us, 5.65 TB/s), and the ten rounds cost about 100 integer
// operations per call, 13 per 16-bit element.  Short calls are at the host call (6.2 us, 2.7 on
// the GPU).  Floats take four
// columns per lane and draw each call's numbers twice, so that a wavefront's accesses stay
// contiguous 16-byte ones.
#include <cmath>

#include "philox.hpp"
#include "rows.hpp"

namespace moe {

struct DropRows {
  const void* x;
  const void* residual;
  void* out;
  int64_t x_stride, residual_stride, out_stride;
  int T, d;
  uint32_t pieces;     // per row
  uint32_t total;      // T * pieces, below 2^31
  uint32_t mul, shift;  // i / pieces = (mulhi(i, mul) + i) >> shift for i < 2^31
  DropDev drop;
};

// One piece of a row (16 bytes), and its elements as floats.
template <typename S, int kN>
__device__ __forceinline__ u32x4_t load_cols(const S* p) {
  if constexpr (sizeof(S) == 2)
    return *(const MOE_GLOBAL u32x4_a2_t*)p;
  else
    return *(const MOE_GLOBAL u32x4_a4_t*)p;
}
template <typename S, int kN>
__device__ __forceinline__ float col_of(const u32x4_t& w, int i) {
  if constexpr (std::is_same<S, float>::value) {
    return __uint_as_float(w[i]);
  } else if constexpr (std::is_same<S, bf16_row_t>::value) {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  } else {
    const uint32_t word = w[i >> 1];
    return (float)__builtin_bit_cast(f16x2_t, word)[i & 1];
  }
}
// A dropped element is selected away, not multiplied by zero: infinities and NaN in it do
// not reach the output.
__device__ __forceinline__ float dropped(float x, bool keep, float scale, float r) {
  return keep ? fmaf(x, scale, r) : r;
}

template <typename S>
__global__ __launch_bounds__(256) void k_dropout(DropRows a) {
  constexpr int kN = sizeof(S) == 2 ? 8 : 4;
  DropKey key{};
  if (a.drop.threshold) key = drop_key(a.drop);
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < a.total; i += step) {
    const uint32_t row = (__umulhi(i, a.mul) + i) >> a.shift;
    const uint32_t col = (i - row * a.pieces) * kN;
    const S* x = static_cast<const S*>(a.x) + (int64_t)row * a.x_stride;
    const S* res = a.residual ? static_cast<const S*>(a.residual) + (int64_t)row * a.residual_stride : nullptr;
    S* out = static_cast<S*>(a.out) + (int64_t)row * a.out_stride;
    u32x4_t n{};
    if (a.drop.threshold) n = drop_numbers(key, a.drop.site, row, col >> 3);
    const int first = kN == 4 ? (int)(col & 4) : 0;  // this lane's first number of the call's eight
    if (col + kN <= (uint32_t)a.d) {
      const u32x4_t w = load_cols<S, kN>(x + col);
      u32x4_t r{};
      if (res) r = load_cols<S, kN>(res + col);
      float v[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const bool keep = kN == 8 ? drop_keeps(n, j, a.drop.threshold)
                                  : (first ? drop_keeps(n, 4 + (j & 3), a.drop.threshold)
                                           : drop_keeps(n, j & 3, a.drop.threshold));
        v[j] = dropped(col_of<S, kN>(w, j), keep, a.drop.scale, col_of<S, kN>(r, j));
      }
      u32x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (std::is_same<S, float>::value)
          o[j] = __float_as_uint(v[j]);
        else if constexpr (std::is_same<S, bf16_row_t>::value)
          o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        else
          o[j] = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)v[2 * j], (_Float16)v[2 * j + 1]});
      }
      if constexpr (sizeof(S) == 2)
        __builtin_nontemporal_store(o, (MOE_GLOBAL u32x4_a2_t*)(out + col));
      else
        __builtin_nontemporal_store(o, (MOE_GLOBAL u32x4_a4_t*)(out + col));
    } else {
      for (int j = 0; col + j < (uint32_t)a.d; ++j) {  // a row's last columns, one at a time
        const bool keep = ((n[(first + j) >> 1] >> (16 * ((first + j) & 1))) & 0xFFFFu) >= a.drop.threshold;
        store_one(out + col + j, dropped(load_one(x + col + j), keep, a.drop.scale, res ? load_one(res + col + j) : 0.f));
      }
    }
  }
}

int check_dropout(const char* fn, double p, const int64_t* state, int site) {
  MOE_CHECK_ARG(p >= 0.0 && p <= 1.0, MOE_ERR_INVALID_ARG, "%s: dropout probability %g outside [0, 1]", fn, p);
  if (p == 0.0) return MOE_OK;
  MOE_CHECK_ARG(state && ((uintptr_t)state % 8) == 0, MOE_ERR_INVALID_ARG, "%s: dropout state is NULL or misaligned", fn);
  MOE_CHECK_ARG(site >= 0 && site < MOE_DROPOUT_SITES, MOE_ERR_INVALID_ARG, "%s: dropout site %d outside [0, %d)", fn,
                site, MOE_DROPOUT_SITES);
  return MOE_OK;
}

DropDev drop_dev(double p, const int64_t* state, int site) {
  DropDev d;
  d.state = state;
  d.threshold = (uint32_t)std::floor(p * 65536.0 + 0.5);
  d.site = d.threshold ? (uint32_t)site << 21 : 0u;
  d.scale = d.threshold < 65536u ? (float)(65536.0 / (65536.0 - d.threshold)) : 0.f;
  return d;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_dropout(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, int dtype,
                           int T, int d, double p, const int64_t* state, int site, void* out, int64_t out_stride,
                           void* stream) {
  clear_error();
  const char* fn = "moe_dropout";
  MOE_CHECK_ARG(dtype >= MOE_BF16 && dtype <= MOE_FP32, MOE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  MOE_CHECK_ARG(T >= 0 && d > 0, MOE_ERR_INVALID_ARG, "%s: bad sizes T=%d d=%d", fn, T, d);
  MOE_CHECK_ARG(d <= (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE, "%s: unsupported d=%d (<= 2^24)", fn, d);
  const int64_t size = dtype_bytes(dtype), per = dtype == MOE_FP32 ? 4 : 8;
  const int64_t pieces = ceil_div(d, per), total = (int64_t)T * pieces;
  MOE_CHECK_ARG(total < (1ll << 31) - (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: unsupported T=%d d=%d (T ceil(d / %d) < 2^31 - 2^24)", fn, T, d, (int)per);
  const int rc = check_dropout(fn, p, state, site);
  if (rc || T == 0) return rc;
  MOE_CHECK_ARG(x && out && ((uintptr_t)x % size) == 0 && ((uintptr_t)out % size) == 0 &&
                    ((uintptr_t)residual % size) == 0,
                MOE_ERR_INVALID_ARG, "%s: x or out is NULL, or a tensor misaligned", fn);
  MOE_CHECK_ARG(x_stride >= 0 && (!residual || residual_stride >= 0) && out_stride >= d, MOE_ERR_INVALID_ARG,
                "%s: negative stride, or out's below %d", fn, d);
  DropRows a{x, residual, out, x_stride, residual_stride, out_stride, T, d, (uint32_t)pieces, (uint32_t)total, 0, 0,
             drop_dev(p, state, site)};
  while ((1ll << a.shift) < pieces) ++a.shift;
  a.mul = (uint32_t)(((uint64_t)((1ll << a.shift) - pieces) << 32) / (uint64_t)pieces + 1);
  hipStream_t s = (hipStream_t)stream;
  const unsigned groups = (unsigned)std::min<int64_t>(ceil_div(total, 256), 1 << 16);
  timing_begin(K_DROPOUT, s);
  with_dtype(dtype, [&](auto e) {
    hipLaunchKernelGGL(k_dropout<decltype(e)>, dim3(groups), dim3(256), 0, s, a);
  });
  timing_end(K_DROPOUT, s);
  return check_launch(fn);
}

// Row tensors of a runtime type (bf16, fp16, fp32) for the row operators (expert-sorted
// rows, block norms): 8-element pieces of a row as floats, and sums over lanes.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace moe {

// timing ids of the row operators, behind those of the grouped passes
enum RowKernelId { K_PERMUTE = K_NUM, K_UNPERMUTE, K_ROUTE_BWD, K_BLOCK_NORM, K_BLOCK_NORM_BWD, K_NUM_ALL };
static_assert(K_PERMUTE == 11, "the ids the header lists");

struct bf16_row_t {
  uint16_t bits;
};
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at the alignment of one element: rows of odd lengths start anywhere, and
// gfx950 reads and writes unaligned global memory in one instruction
typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));

inline int64_t dtype_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

constexpr int kPiece = 8;  // elements of a row that one lane holds at a time

// Eight consecutive elements as they lie in memory.
template <typename S>
struct Raw {
  u32x4_t w[sizeof(S) == 4 ? 2 : 1];
};

__device__ __forceinline__ float to_f32(bf16_row_t v) { return bf16_bits_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(bf16_row_t* p, float v) { p->bits = (uint16_t)f32_to_bf16_bits(v); }
__device__ __forceinline__ void from_f32(_Float16* p, float v) { *p = (_Float16)v; }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }

// elements [0, n) of a piece of which n are in the row; the rest reads as zero
template <typename S>
__device__ __forceinline__ Raw<S> load_raw(const S* p, int n) {
  Raw<S> r;
  if (n >= kPiece) {
    if constexpr (sizeof(S) == 2) {
      r.w[0] = *reinterpret_cast<const u32x4_a2_t*>(p);
    } else {
      r.w[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
      r.w[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
    }
  } else {
    if constexpr (sizeof(S) == 2) {
      uint32_t h[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) h[i] = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[0][i] = h[2 * i] | (h[2 * i + 1] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) r.w[i >> 2][i & 3] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    }
  }
  return r;
}

template <typename S>
__device__ __forceinline__ void store_raw(S* p, const Raw<S>& r, int n) {
  if (n >= kPiece) {
    if constexpr (sizeof(S) == 2) {
      *reinterpret_cast<u32x4_a2_t*>(p) = r.w[0];
    } else {
      *reinterpret_cast<u32x4_a4_t*>(p) = r.w[0];
      *reinterpret_cast<u32x4_a4_t*>(p + 4) = r.w[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      if constexpr (sizeof(S) == 2) {
        if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(r.w[0][i >> 1] >> (16 * (i & 1)));
      } else {
        if (i < n) reinterpret_cast<uint32_t*>(p)[i] = r.w[i >> 2][i & 3];
      }
    }
  }
}

template <typename S>
__device__ __forceinline__ void unpack(const Raw<S>& r, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    if constexpr (std::is_same<S, float>::value) {
      v[i] = __uint_as_float(r.w[i >> 2][i & 3]);
    } else if constexpr (std::is_same<S, bf16_row_t>::value) {
      v[i] = __uint_as_float((i & 1) ? (r.w[0][i >> 1] & 0xFFFF0000u) : (r.w[0][i >> 1] << 16));
    } else {
      const uint32_t w = r.w[0][i >> 1];  // a value of its own: a cast of the vector's element takes element 0
      v[i] = (float)__builtin_bit_cast(f16x2_t, w)[i & 1];
    }
  }
}

// one rounding to the row's type, to nearest even
template <typename S>
__device__ __forceinline__ Raw<S> pack(const float (&v)[kPiece]) {
  Raw<S> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<S, float>::value) {
      r.w[0][i] = __float_as_uint(v[i]);
      r.w[1][i] = __float_as_uint(v[4 + i]);
    } else if constexpr (std::is_same<S, bf16_row_t>::value) {
      r.w[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
      r.w[0][i] = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    }
  }
  return r;
}

template <typename S>
__device__ __forceinline__ void load_piece(const S* p, int n, float (&v)[kPiece]) {
  unpack<S>(load_raw(p, n), v);
}
template <typename S>
__device__ __forceinline__ void store_piece(S* p, int n, const float (&v)[kPiece]) {
  store_raw(p, pack<S>(v), n);
}

// Calls f with a value of the row type of `dtype` (checked by the caller).
template <typename F>
void with_dtype(int dtype, F&& f) {
  if (dtype == MOE_BF16)
    f(bf16_row_t{});
  else if (dtype == MOE_FP16)
    f(_Float16{});
  else
    f(float{});
}

}  // namespace moe

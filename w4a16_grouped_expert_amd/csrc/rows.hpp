// Row tensors of a runtime type (bf16, fp16, fp32) for the row operators (expert-sorted
// rows, block norms): 8-element pieces of a row as floats, and sums over lanes.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace moe {

// timing ids of the row operators, behind those of the grouped passes
enum RowKernelId { K_PERMUTE = K_NUM, K_UNPERMUTE, K_ROUTE_BWD, K_BLOCK_NORM, K_BLOCK_NORM_BWD, K_GATED_FFN,
                   K_GATED_FFN_BWD, K_DROPOUT, K_NUM_ALL };
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
// T*d of a call: a lane per piece, rows filled up to whole wavefronts, stays below the 2^32
// threads that a launch may have
constexpr int64_t kMaxRowElements = (int64_t)1 << 34;

// Eight consecutive elements as they lie in memory.
template <typename S>
struct Raw {
  u32x4_t w[sizeof(S) == 4 ? 2 : 1];
};

// Where a lane's eight elements of a row of d lie.  The last piece of a row whose length
// is no multiple of 8 starts at d - 8, and so do those of lanes past the end: every load
// and store is one of eight elements inside the row, and none sits under a branch.  The
// first `skip` elements of such a piece belong to pieces before it.  They are left out of
// sums (mask_piece); outputs are computed and stored twice, the same bits both times.
// kTiny: rows of fewer than eight elements too (at = 0, element by element, skip = 0 for
// the first lane); kernels take it for short rows only.
struct Piece {
  uint32_t at;  // first element
  int skip;
};
__device__ __forceinline__ Piece piece_of(int col, int d) {
  const int at = col + kPiece <= d ? col : d > kPiece ? d - kPiece : 0;
  return {(uint32_t)at, col - at < kPiece ? col - at : kPiece};
}
// (Global memory by a scalar base and a 32-bit offset in bytes where the row's address is
// uniform: no vector registers for addresses.  The asm keeps the offset's extension to 64
// bits beside the access, where the compiler can see that it needs none.)
#define MOE_GLOBAL __attribute__((address_space(1)))
template <typename S>
__device__ __forceinline__ uint32_t piece_offset(const Piece& p) {
  uint32_t o = p.at * (uint32_t)sizeof(S);
  asm volatile("" : "+v"(o));
  return o;
}
template <typename S>
__device__ __forceinline__ const MOE_GLOBAL char* piece_ptr(const S* row, const Piece& p) {
  return (const MOE_GLOBAL char*)row + piece_offset<S>(p);
}
template <typename S>
__device__ __forceinline__ MOE_GLOBAL char* piece_ptr(S* row, const Piece& p) {
  return (MOE_GLOBAL char*)row + piece_offset<S>(p);
}

// kStream: non-temporal.
template <bool kTiny, bool kStream = false, typename S>
__device__ __forceinline__ Raw<S> load_raw(const S* row, const Piece& p, int d) {
  Raw<S> r;
  if (!kTiny || d >= kPiece) {
    const MOE_GLOBAL char* q = piece_ptr(row, p);
    if constexpr (sizeof(S) == 2 && kStream) {
      r.w[0] = __builtin_nontemporal_load((const MOE_GLOBAL u32x4_a2_t*)q);
    } else if constexpr (sizeof(S) == 2) {
      r.w[0] = *(const MOE_GLOBAL u32x4_a2_t*)q;
    } else if constexpr (kStream) {
      r.w[0] = __builtin_nontemporal_load((const MOE_GLOBAL u32x4_a4_t*)q);
      r.w[1] = __builtin_nontemporal_load((const MOE_GLOBAL u32x4_a4_t*)(q + 16));
    } else {
      r.w[0] = *(const MOE_GLOBAL u32x4_a4_t*)q;
      r.w[1] = *(const MOE_GLOBAL u32x4_a4_t*)(q + 16);
    }
  } else {
    uint32_t h[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const int e = i < d ? i : 0;
      if constexpr (sizeof(S) == 2)
        h[i] = reinterpret_cast<const uint16_t*>(row)[e];
      else
        h[i] = reinterpret_cast<const uint32_t*>(row)[e];
      h[i] = i < d ? h[i] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      if constexpr (sizeof(S) == 2)
        r.w[0][i >> 1] = (i & 1) ? r.w[0][i >> 1] | (h[i] << 16) : h[i];
      else
        r.w[i >> 2][i & 3] = h[i];
    }
  }
  return r;
}

// zero for the elements that are not this piece's (at the first use, not at the load)
template <typename S>
__device__ __forceinline__ void mask_piece(Raw<S>& r, const Piece& p) {
  if (p.skip) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      if constexpr (sizeof(S) == 2)
        r.w[0][i >> 1] &= i < p.skip ? ((i & 1) ? 0x0000FFFFu : 0xFFFF0000u) : 0xFFFFFFFFu;
      else
        r.w[i >> 2][i & 3] = i < p.skip ? 0u : r.w[i >> 2][i & 3];
    }
  }
}

// Rows are stored past the L2 (non-temporal): what a launch leaves dirty there is written
// back at its end, when nothing else runs (permute at T = 4096, d = 2048, k = 8: 30.5 to
// 26.3 us, block norm gradient 43.8 to 40.3; small calls unchanged).  kStream = false: plain
// stores, for what the next launch reads.
template <bool kTiny, bool kStream = true, typename S>
__device__ __forceinline__ void store_raw(S* row, const Piece& p, int d, const Raw<S>& r) {
  if (!kTiny || d >= kPiece) {
    MOE_GLOBAL char* q = piece_ptr(row, p);
    if constexpr (sizeof(S) == 2 && kStream) {
      __builtin_nontemporal_store(r.w[0], (MOE_GLOBAL u32x4_a2_t*)q);
    } else if constexpr (sizeof(S) == 2) {
      *(MOE_GLOBAL u32x4_a2_t*)q = r.w[0];
    } else if constexpr (kStream && !kTiny) {
      // (the whole wavefront has one row.)  32 lanes' pieces per instruction, both halves of
      // each, so that it fills whole lines: the lower lanes' second halves change places with
      // the upper lanes' first ones.  Without, T = 4096, d = 2048, k = 8: permute 121 in place
      // of 53 us, its gradient's rows 122 in place of 111
      const uint32_t at = piece_offset<S>(p);
      const u32x2_t o = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(at, at + 16, false, false));
      u32x4_t lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = r.w[0][i], b = r.w[1][i];
        const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(a, b, false, false));
        lo[i] = v[0];
        hi[i] = v[1];
      }
      __builtin_nontemporal_store(lo, (MOE_GLOBAL u32x4_a4_t*)((MOE_GLOBAL char*)row + o[0]));
      __builtin_nontemporal_store(hi, (MOE_GLOBAL u32x4_a4_t*)((MOE_GLOBAL char*)row + o[1]));
    } else if constexpr (kStream) {
      __builtin_nontemporal_store(r.w[0], (MOE_GLOBAL u32x4_a4_t*)q);
      __builtin_nontemporal_store(r.w[1], (MOE_GLOBAL u32x4_a4_t*)(q + 16));
    } else {
      *(MOE_GLOBAL u32x4_a4_t*)q = r.w[0];
      *(MOE_GLOBAL u32x4_a4_t*)(q + 16) = r.w[1];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    if (p.skip || i >= d) continue;
    MOE_GLOBAL char* q = (MOE_GLOBAL char*)row + i * sizeof(S);
    if constexpr (sizeof(S) == 2)
      *(MOE_GLOBAL uint16_t*)q = (uint16_t)(r.w[0][i >> 1] >> (16 * (i & 1)));
    else
      *(MOE_GLOBAL uint32_t*)q = r.w[i >> 2][i & 3];
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
__device__ __forceinline__ float load_one(const S* p) {
  if constexpr (std::is_same<S, bf16_row_t>::value)
    return bf16_bits_to_f32(*(const MOE_GLOBAL uint16_t*)p);
  else
    return (float)*(const MOE_GLOBAL S*)p;
}

template <typename S>
__device__ __forceinline__ void store_one(S* p, float v) {
  if constexpr (std::is_same<S, bf16_row_t>::value)
    p->bits = (uint16_t)f32_to_bf16_bits(v);
  else
    *p = (S)v;
}

template <bool kTiny, bool kStream = true, typename S>
__device__ __forceinline__ void store_piece(S* row, const Piece& p, int d, const float (&v)[kPiece]) {
  store_raw<kTiny, kStream>(row, p, d, pack<S>(v));
}

// Row t of a tensor.  A wavefront with one row (not kSub) keeps its address in scalar
// registers, as the base that 32-bit lane offsets add to; left alone the compiler adds the
// lane's offset to the tensor's address first, two vector registers per tensor and piece.
template <typename P>
__device__ __forceinline__ P uniform_ptr(P p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<P>(((uint64_t)hi << 32) | lo);
}
template <typename S, bool kSub>
__device__ __forceinline__ const S* row_ptr(const void* p, int64_t t, int64_t stride) {
  const S* r = static_cast<const S*>(p) + t * stride;
  return kSub ? r : uniform_ptr(r);
}
template <typename S, bool kSub>
__device__ __forceinline__ S* row_ptr(void* p, int64_t t, int64_t stride) {
  S* r = static_cast<S*>(p) + t * stride;
  return kSub ? r : uniform_ptr(r);
}

template <typename S>
__device__ __forceinline__ Raw<S> masked(Raw<S> r, uint32_t mask) {
#pragma unroll
  for (int q = 0; q < (int)(sizeof(r.w) / sizeof(r.w[0])); ++q) r.w[q] &= mask;
  return r;
}

template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, true));
}

// Sum over groups of 1 << lt lanes (lt uniform, 0..6), the same bits in each of its
// lanes: both sides of every step add the same two values.  One vector instruction for
// each of the first four steps (lane ^ 1, ^ 2, and mirrors within 8 and 16 lanes), a swap
// of rows of 16 or halves of 32 and an addition for the last two.
__device__ __forceinline__ float lane_sum(float v, int lt) {
  if (lt > 0) v = add_dpp<0xB1>(v);   // quad_perm 1,0,3,2
  if (lt > 1) v = add_dpp<0x4E>(v);   // quad_perm 2,3,0,1
  if (lt > 2) v = add_dpp<0x141>(v);  // row_half_mirror
  if (lt > 3) v = add_dpp<0x140>(v);  // row_mirror
  if (lt > 4) {
    const uint32_t b = __float_as_uint(v);
    const u32x2_t s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(b, b, false, false));
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (lt > 5) {
    const uint32_t b = __float_as_uint(v);
    const u32x2_t s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
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

// Dropout from a counter-based generator: which elements of a tensor are kept is a function
// of (seed, step, site, row, column) alone, so the gradient draws the same mask again and no
// mask is stored.
//
// Philox-4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): one call gives the eight 16-bit numbers of eight consecutive
// columns.  An element is kept where its number is at least round(p 2^16).
#pragma once

#include "common.hpp"

namespace moe {

struct DropDev {
  const int64_t* state;  // {seed, step} in device memory, so that a replayed graph draws new masks
  uint32_t site;         // which use of the step, << 21: above the column's eighth
  uint32_t threshold;    // 0 .. 65536; 0 keeps everything
  float scale;           // 1 / (1 - threshold / 65536), 0 where nothing is kept
};

// the key and the step as scalars (uniform loads)
struct DropKey {
  uint32_t k0, k1, s0, s1;
};
__device__ __forceinline__ DropKey drop_key(const DropDev& d) {
  const uint64_t seed = (uint64_t)d.state[0], step = (uint64_t)d.state[1];
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step, (uint32_t)(step >> 32)};
}

// The eight numbers of columns 8 block .. 8 block + 7 of a row, two to a word, low halves first.
__device__ __forceinline__ u32x4_t drop_numbers(const DropKey& key, uint32_t site, uint32_t row, uint32_t block) {
  uint32_t c0 = block | site, c1 = row, c2 = key.s0, c3 = key.s1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

__device__ __forceinline__ bool drop_keeps(const u32x4_t& numbers, int i, uint32_t threshold) {
  const uint32_t w = numbers[i >> 1];
  return ((i & 1) ? w >> 16 : w & 0xFFFFu) >= threshold;
}

// Host: the arguments of a call's dropout, checked; p = 0 needs no state.
int check_dropout(const char* fn, double p, const int64_t* state, int site);
DropDev drop_dev(double p, const int64_t* state, int site);

}  // namespace moe

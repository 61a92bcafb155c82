// Products of 16-bit matrices on the matrix cores, C[m][n] = sum_k A(m, k) B(n, k) with
// float32 sums, tiled for one workgroup of eight wavefronts: 128 or 256 m by 256 n.
//
// Either operand may have its k or its m (n) contiguous in memory.  A K step of 64 is staged in
// LDS by DMA (buffer_load ... lds, no registers), two steps deep: while one is multiplied the
// next one lands.
//  - k contiguous: rows of 64 k, 128 bytes; 16-byte chunk c of row r at slot c ^ (r & 7), so
//    that the eight lanes of a phase of ds_read_b128 hit eight different chunks.
//  - m contiguous: rows of one k; 32-byte pair p of row k at slot p ^ (k & 3 | (k >> 1) & 4).
//    ds_read_b64_tr_b16 reads four k by 16 m per 16 lanes and hands each lane the four k of its
//    m, which is half of an MFMA operand; the rows of one instruction hit different pairs.
// Bounds are the buffer resource's: what lies past a tensor, an expert's rows or the K range
// reads as zero.  n enters as the first MFMA operand, so that a lane holds four consecutive n
// of one m, eight after an exchange between lanes: 16-byte stores.
#pragma once

#include "rows.hpp"

namespace moe {

constexpr int kTileN = 256;       // n per workgroup
constexpr int kStepK = 64;        // k per stage
constexpr int kTileWaves = 8;     // 2 in m (rows of 16 in turn) x 4 in n (64 each)
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kNI = 4;            // 16-column blocks of a wavefront
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every resource

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
#define MOE_LDS __attribute__((address_space(3)))

template <typename S>
__device__ __forceinline__ f32x4_t mfma16(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
  if constexpr (std::is_same<S, bf16_row_t>::value)
    return mfma16x16x32(as_bf16x8(a), as_bf16x8(b), c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// 16 bytes per lane from a buffer resource to LDS at lds + 16 lane.  The compiler neither
// counts these loads nor knows what they write: every reader waits for them itself
// (stage_barrier below).
__device__ __forceinline__ void dma16(const i32x4_t& rsrc, uint32_t offset, uint32_t lds) {
  uint32_t saved;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(saved) : "v"(offset), "s"(rsrc), "s"(lds) : "memory");
}
// This wavefront's DMA has landed and its LDS reads are done; then the workgroup's.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ i32x4_t resource(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)((a >> 32) & 0xFFFF)),
                 __builtin_amdgcn_readfirstlane((int)bytes), kBufferRsrcWord3};
}

// One operand of a tile: where its elements lie.
struct OperandTile {
  const char* base;  // element (m0, k = 0)
  int ld;            // elements between rows (of k, or of m where m is contiguous)
  int rows;          // m that are there from m0 on (at least 1)
};

// The staging of one operand of kX m (a multiple of 128) by the wavefronts of a workgroup.
// kDual: two tensors of kX / 2 rows each, one behind the other in the stage (k contiguous).
template <int kX, bool kMContig, bool kDual = false>
struct Stager {
  static constexpr int kBytes = kX * kStepK * 2;
  static constexpr int kIssues = kBytes / 1024 / kTileWaves;  // DMA instructions per wavefront and step
  static_assert(!(kMContig && kDual), "two tensors lie one behind the other with k contiguous only");
  const char* base;
  int ld2;           // bytes between rows
  int rows;
  int K;
  uint32_t off[2];   // this lane's offset; m contiguous: of even and odd instructions
  int kc8;           // k contiguous: first k of this lane's chunk
  uint32_t bytes;    // k contiguous: size of the resource

  // t: the operand's tile; for kDual t2 is the second tensor's
  __device__ __forceinline__ void start(const OperandTile& t, int k_total, int wave, int lane,
                                        const OperandTile* t2 = nullptr) {
    const OperandTile& mine = kDual && wave >= kTileWaves / 2 ? *t2 : t;
    base = mine.base;
    ld2 = mine.ld * 2;
    rows = mine.rows;
    K = k_total;
    if constexpr (!kMContig) {
      // instruction j of a wavefront fills rows 8 (wave kIssues + j) .. + 7: lane l the slot l & 7 of row l >> 3
      const int first = 8 * kIssues * (kDual ? wave & (kTileWaves / 2 - 1) : wave) + (lane >> 3);
      kc8 = 8 * ((lane & 7) ^ (lane >> 3));
      off[0] = (uint32_t)first * (uint32_t)ld2 + 2u * kc8;
      const int there = rows < (kDual ? kX / 2 : kX) ? rows : (kDual ? kX / 2 : kX);
      bytes = (uint32_t)(there - 1) * (uint32_t)ld2 + 2u * K;
    } else {
      constexpr int kChunks = kX / 8, kRows = 64 / kChunks;  // 16-byte chunks per row, rows per instruction
      const int pos = lane & (kChunks - 1);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int k = (wave * kIssues + v) * kRows + lane / kChunks;
        const int s = (k & 3) | ((k >> 1) & 4);
        off[v] = (uint32_t)k * (uint32_t)ld2 + 16u * (pos ^ (2 * s));
      }
    }
  }
  // stage the step that starts at k0 (a multiple of kStepK below K)
  __device__ __forceinline__ void issue(int k0, uint32_t lds, int wave) const {
    const uint32_t to = lds + wave * kIssues * 1024;
    if constexpr (!kMContig) {
      const i32x4_t r = resource(base, bytes);
      const uint32_t from = k0 + kc8 < K ? off[0] + 2u * k0 : kOutside;
#pragma unroll
      for (int j = 0; j < kIssues; ++j) dma16(r, from + (uint32_t)(8 * j * ld2), to + 1024 * j);
    } else {
      constexpr int kRows = 64 / (kX / 8);
      static_assert(kIssues * kRows == 8, "the k of a wavefront's instructions: 8 wave .. + 7");
      const int left = K - k0 < kStepK ? K - k0 : kStepK;
      const i32x4_t r = resource(base + (int64_t)k0 * ld2, (uint32_t)(left - 1) * (uint32_t)ld2 + 2u * rows);
#pragma unroll
      for (int j = 0; j < kIssues; ++j) dma16(r, off[j & 1] + (uint32_t)((j & ~1) * kRows * ld2), to + 1024 * j);
    }
  }
};

// This lane's MFMA operands of a staged operand: 16-m block b (of the kX / 16), k 32 s .. + 31.
template <int kX, bool kMContig>
struct Reader {
  uint32_t at[kMContig ? 4 : 2];
  // first: the lane's first block; blocks follow at a step of kStride blocks
  __device__ __forceinline__ void start(int first, int stride, int lane) {
    const int i = lane & 15, q = lane >> 4;
    if constexpr (!kMContig) {
#pragma unroll
      for (int s = 0; s < 2; ++s) at[s] = (uint32_t)((first * 16 + i) * 128 + 16 * ((4 * s + q) ^ (i & 7)));
    } else {
      const int k = 8 * q + (i >> 2), s = (k & 3) | ((k >> 1) & 4);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        at[v] = (uint32_t)(k * kX * 2 + 32 * ((first + v * stride) ^ s) + 8 * (i & 3));
    }
  }
  // k contiguous: the block `blocks` behind the lane's first one; m contiguous: the lane's
  // block number `blocks`, with kStride blocks between two (1: of four, 2: of eight).  s: half of the step.
  template <int kStride>
  __device__ __forceinline__ u32x4_t get(const char* stage, int blocks, int s) const {
    if constexpr (!kMContig) {
      return *reinterpret_cast<const u32x4_t*>(stage + at[s] + blocks * 2048);
    } else {
      // (blocks 4 and up lie eight pairs behind 0 to 3)
      const char* p = stage + at[blocks & 3] + (blocks >> 2) * 256 + s * (32 * kX * 2);
      typedef MOE_LDS s16x4_t* lds_ptr;
      const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
      const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * kX * 2)));
      return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

// Eight consecutive columns of one row from two neighbouring 16-column blocks of a
// wavefront's results: lane 16 q + i has columns 4 q .. 4 q + 3 of both blocks in row i, and
// ends up with columns 0, 16, 8 or 24 (q = 0 .. 3) and the seven behind.
__device__ __forceinline__ int eight_column(int lane) { return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8; }
__device__ __forceinline__ void eight_columns(const f32x4_t& a, const f32x4_t& b, float (&v)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t x = __float_as_uint(a[r]), y = __float_as_uint(b[r]);
    const u32x2_t s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(x, y, false, false));
    v[r] = __uint_as_float(s[0]);
    v[4 + r] = __uint_as_float(s[1]);
  }
}

}  // namespace moe

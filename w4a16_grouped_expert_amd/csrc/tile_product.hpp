// Products of 16-bit matrices on the matrix cores, C[m][n] = sum_k A(m, k) B(n, k) with
// float32 sums, by tiles of up to 256 m by 256 n per workgroup.
//
// Either operand may have its k or its m (n) contiguous in memory.  Units of 64 k are staged
// in a ring in LDS by DMA (buffer_load ... lds, no registers), ahead of the products and across
// the tiles of a workgroup: the first units of a tile land while the tile before it is stored.
// Each wavefront reads the operands of one half of a unit into registers while it multiplies
// the half before.
//  - k contiguous: rows of 64 k, 128 bytes, whole cache lines (rows of 64 bytes come at half the
//    rate: 70 against 130 GB/s per CU out of the L2); 16-byte chunk c of row r at slot c ^ (r & 7),
//    so that the lanes of a phase of ds_read_b128 hit different banks.
//  - m contiguous: rows of one k; 32-byte pair p of row k at slot p ^ pair_swizzle(k).
//    ds_read_b64_tr_b16 reads four k by 16 m per 16 lanes and hands each lane the four k of its
//    m, which is half of an MFMA operand; the rows of one instruction hit different pairs.
// Bounds are the buffer resource's: what lies past a tensor, an expert's rows or the K range
// reads as zero.  n enters as the first MFMA operand, so that a lane holds four consecutive n
// of one m, eight after an exchange between lanes: 16-byte stores.
#pragma once

#include "rows.hpp"

namespace moe {

constexpr int kUnitK = 64;  // k per unit, two MFMA steps
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
// (stage_barrier below).  Nor does it keep their distances: a vector instruction that writes the
// resource (v_readfirstlane, a scalar register that comes back from a lane) has to lie five wait
// states in front of the load, one of s_mov and four of s_nop.  M0 is declared as written: what
// else reads it sets it again.
__device__ __forceinline__ void dma16(const i32x4_t& rsrc, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(offset), "s"(rsrc), "s"(lds) : "memory", "m0");
}
// At most kPending of this wavefront's vector memory operations are in flight (they end in
// order) and its LDS reads are done; then the workgroup meets.
template <int kPending>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kPending) : "memory");
}
// Loads and stores of an epilogue through a resource of 2^31 - 1 bytes: kOutside reads zero
// and stores nothing, so that every lane executes every one of them.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t open_resource(const void* base) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), 0, 0x7FFFFFFF,
                                           kBufferRsrcWord3);
}
template <int kPolicy = 0>
__device__ __forceinline__ void store16(const u32x4_t& v, __amdgpu_buffer_rsrc_t r, uint32_t offset) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, offset, 0, kPolicy);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0);
}
__device__ __forceinline__ int pair_swizzle(int k) { return (k & 3) | ((k >> 1) & 4); }
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

// The staging of one operand of kX m (64, 128 or 256) by the kWaves wavefronts of a workgroup,
// one unit after the other.
// kDual: two tensors of kX / 2 rows each, one behind the other in the stage (k contiguous).
template <int kX, int kWaves, bool kMContig, bool kDual = false>
struct Stager {
  static constexpr int kBytes = kX * kUnitK * 2;
  static constexpr int kIssues = kBytes / 1024 / kWaves;  // DMA instructions per wavefront and unit
  static constexpr int kChunks = kX / 8;                  // m contiguous: 16-byte chunks of a row,
  static constexpr int kRows = 64 / kChunks;              // rows of k per instruction
  static_assert(!(kMContig && kDual), "two tensors lie one behind the other with k contiguous only");
  static_assert(kIssues * kWaves * 1024 == kBytes, "");
  const char* base;  // m contiguous: moves on with the units
  int ld2;           // bytes between rows
  int left;          // k from the next unit on
  uint32_t edge;     // k contiguous: size of the resource; m contiguous: bytes of a row
  uint32_t off[kMContig ? kIssues : 1];  // this lane's offset in the next unit; m contiguous: of each instruction
  int kc8;           // k contiguous: first k of this lane's chunk within a unit

  // t: the operand's tile; for kDual t2 is the second tensor's
  __device__ __forceinline__ void start(const OperandTile& t, int k_total, int wave, int lane,
                                        const OperandTile* t2 = nullptr) {
    const OperandTile& mine = kDual && wave >= kWaves / 2 ? *t2 : t;
    base = mine.base;
    ld2 = mine.ld * 2;
    left = k_total;
    if constexpr (!kMContig) {
      // instruction j of a wavefront fills 8 rows from 8 (wave kIssues + j): lane l the slot l & 7 of row l >> 3
      const int first = 8 * kIssues * (kDual ? wave & (kWaves / 2 - 1) : wave) + (lane >> 3);
      kc8 = 8 * ((lane & 7) ^ (lane >> 3));
      off[0] = (uint32_t)first * (uint32_t)ld2 + 2u * kc8;
      edge = __builtin_amdgcn_readfirstlane((min(mine.rows, kDual ? kX / 2 : kX) - 1) * ld2 + 2 * k_total);
    } else {
      const int pos = lane & (kChunks - 1);
#pragma unroll
      for (int j = 0; j < kIssues; ++j) {
        const int k = (wave * kIssues + j) * kRows + lane / kChunks;
        off[j] = (uint32_t)k * (uint32_t)ld2 + 16u * (pos ^ (2 * pair_swizzle(k)));
      }
      edge = 2u * mine.rows;
    }
  }
  // nothing more to stage: the units from here on are zeros
  __device__ __forceinline__ void stop() { left = 0; }
  // instruction j (a constant, in order) of the staging of the next unit; the last one moves on
  __device__ __forceinline__ void issue(int j, uint32_t lds, int wave) {
    const uint32_t to = lds + (wave * kIssues + j) * 1024;
    if constexpr (!kMContig) {
      const uint32_t from = kc8 < left ? off[0] : kOutside;
      dma16(resource(base, edge), from + (uint32_t)(8 * j * ld2), to);
    } else {
      const i32x4_t r = resource(base, left > 0 ? (uint32_t)(min(left, kUnitK) - 1) * (uint32_t)ld2 + edge : 0u);
      dma16(r, off[j], to);
    }
    if (j + 1 < kIssues) return;
    if constexpr (!kMContig)
      off[0] += 2 * kUnitK;
    else
      base += (int64_t)kUnitK * ld2;
    left -= kUnitK;
  }
};

// This lane's MFMA operands of a staged operand: blocks of 16 m, kStride between two of them.
template <int kX, bool kMContig, int kStride>
struct Reader {
  uint32_t at[2];  // of the two halves of a unit
  __device__ __forceinline__ void start(int first, int lane) {
    const int i = lane & 15, q = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (!kMContig) {
        at[s] = (uint32_t)((first * 16 + i) * 128 + 16 * ((4 * s + q) ^ (i & 7)));
      } else {
        const int k = 32 * s + 8 * q + (i >> 2);
        at[s] = (uint32_t)(k * kX * 2 + 32 * (first ^ pair_swizzle(k)) + 8 * (i & 3));
      }
    }
  }
  // block b (a constant) of half s of the operand staged at `stage` in LDS.  m contiguous: the pair
  // of block b is that of block 0 with bits changed that are zero in the first block's number.
  __device__ __forceinline__ u32x4_t get(uint32_t stage, int b, int s) const {
    if constexpr (!kMContig) {
      return *reinterpret_cast<const MOE_LDS u32x4_t*>((uintptr_t)(stage + at[s] + b * kStride * 2048));
    } else {
      const uintptr_t p = ((stage + at[s]) ^ (((b * kStride) & 7) * 32)) + ((b * kStride) >> 3) * 256;
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

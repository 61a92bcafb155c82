// moe_route_backward: from the gradient of the routing weights to those of the router's
// input and weight (ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient
// W4A16 Inference", Abstract: BF16 router, unchanged top-k).
//
// With G [T][E] the gradient of the logits, dx = G W (+ dx_add) and dW = G^T x.  W and x
// are bf16 as they are; G is split into bf16 parts whose sum is G to 2^-18 (two parts,
// for dx, which is rounded to bf16) or 2^-27 (three parts, for the float32 dW), so both
// products run on the bf16 matrix cores with float32 sums.
//
// Both products contract over the rows of a row-major bf16 matrix (W over e, x over t).
// A 16x16x32 MFMA wants eight consecutive k per lane: a lane loads eight rows of its 16
// bytes (eight columns), and v_perm pairs the rows, which transposes the 8 x 8 block in
// registers.  MFMA i of eight then has column 8n + i as its column n, so a lane ends with
// eight consecutive columns of the result.
//
// G itself: with the softmax over the selected experts and no loss on the logits it has k
// values per token, and each wavefront builds the 32-token tiles it needs in its part of
// LDS from the pairs; otherwise a first launch writes G in float32 and the tiles are read.
#include "rows.hpp"

namespace moe {

constexpr int kRbCols = 128;   // columns of d per wavefront
constexpr int kRbWaves = 8;    // wavefronts per workgroup of the products
constexpr int kRbTile = 64;    // experts of a tile of G for dx (32 for dW)
constexpr int tile_ld(int kE) { return kE + 4; }  // floats per token of a tile: rows stay 16-byte aligned
static_assert(MOE_MAX_TOPK <= 16, "a lane holds every other pair of its token, at most eight");

struct RouteBackDev {
  const uint16_t *x, *w;
  int T, d, E, k, renormalize;
  int64_t Tp;  // T rounded up to 32
  int Ep;      // E rounded up to 64
  const float* logits;
  const int32_t* ids;
  const float *weights, *dweights, *dlogits;
  const uint16_t* dx_add;
  uint16_t* dx;
  float* dw;
  float* g;     // [Tp][Ep] G, or null: built from the pairs
  float* part;  // [splits][E][d] or null
  int splits;
};

// G of four tokens, a wavefront each, its E <= 64 kEL logits (read once) in the lanes'
// registers.
template <int kEL>
__global__ __launch_bounds__(256) void k_route_dlogits(RouteBackDev a) {
  const int lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  float v[kEL];
#pragma unroll
  for (int i = 0; i < kEL; ++i) v[i] = 0.f;
  if (t < a.T) {
    float add[kEL];
#pragma unroll
    for (int i = 0; i < kEL; ++i) {
      const int e = lane + 64 * i;
      v[i] = !a.renormalize && e < a.E ? a.logits[t * a.E + e] : -INFINITY;
      add[i] = a.dlogits && e < a.E ? a.dlogits[t * a.E + e] : 0.f;
    }
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (lane < a.k) {
      id = a.ids[t * a.k + lane];
      w = a.weights[t * a.k + lane];
      dw = a.dweights[t * a.k + lane];
      if (id < 0 || id >= a.E) {
        id = -1;
        w = dw = 0.f;
      }
    }
    const float s = lane_sum(w * dw, 6);
    if (a.renormalize) {
#pragma unroll
      for (int i = 0; i < kEL; ++i) v[i] = 0.f;
    } else {
      float top = v[0], sum = 0.f;
#pragma unroll
      for (int i = 1; i < kEL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
#pragma unroll
      for (int i = 0; i < kEL; ++i) {
        v[i] = expf(v[i] - top);  // 0 past the last expert
        sum += v[i];
      }
      sum = lane_sum(sum, 6);
#pragma unroll
      for (int i = 0; i < kEL; ++i) v[i] = -(v[i] / sum) * s;
    }
    // the selected experts' own values, to the lanes that hold them
    const float own = w * (dw - s);
    for (int j = 0; j < a.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own), j));
#pragma unroll
      for (int i = 0; i < kEL; ++i) v[i] = e == lane + 64 * i ? o : v[i];
    }
#pragma unroll
    for (int i = 0; i < kEL; ++i) v[i] += add[i];
  }
#pragma unroll
  for (int i = 0; i < kEL; ++i)
    if (lane + 64 * i < a.Ep) a.g[t * a.Ep + lane + 64 * i] = v[i];
}

// What a wavefront needs to build tiles of 32 tokens: two lanes per token, each with
// every other of its pairs.  The tokens' pairs lie one after the other: they are loaded
// in that order (whole cache lines) and dealt out through the wavefront's tile.
// (LDS operations of one wavefront take effect in order.)
struct TilePairs {
  int id[8];
  float g[8];
};
struct PairLoads {
  int id[8];
  float w[8], g[8];
};
__device__ __forceinline__ PairLoads request_pairs(const RouteBackDev& a, int64_t t0) {
  PairLoads r;
  const int64_t base = t0 * a.k, last = (int64_t)a.T * a.k - 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i >= a.k) break;  // (32 k pairs)
    int64_t at = base + 64 * i + lane_id();
    at = at < last ? at : last;
    r.id[i] = a.ids[at];
    r.w[i] = a.weights[at];
    r.g[i] = a.dweights[at];
  }
  return r;
}
__device__ __forceinline__ TilePairs deal_pairs(const RouteBackDev& a, const PairLoads& r, int64_t t0, float* tile) {
  const int lane = lane_id();
  float* stage_w = tile + 32 * MOE_MAX_TOPK;
  float* stage_g = stage_w + 32 * MOE_MAX_TOPK;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i >= a.k) break;
    tile[64 * i + lane] = __int_as_float(r.id[i]);
    stage_w[64 * i + lane] = r.w[i];
    stage_g[64 * i + lane] = r.g[i];
  }
  __builtin_amdgcn_wave_barrier();
  TilePairs p;
  const bool live = t0 + (lane >> 1) < a.T;
  float w[8], s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.id[i] = -1;
    w[i] = p.g[i] = 0.f;
    if (2 * i >= a.k) continue;
    const int j = (lane & 1) + 2 * i, at = (lane >> 1) * a.k + (j < a.k ? j : 0);
    const int id = __float_as_int(tile[at]);
    const bool there = live && j < a.k && id >= 0 && id < a.E;
    p.id[i] = there ? id : -1;
    w[i] = there ? stage_w[at] : 0.f;
    p.g[i] = there ? stage_g[at] : 0.f;
    s = fmaf(w[i], p.g[i], s);
  }
  s = lane_sum(s, 1);
#pragma unroll
  for (int i = 0; i < 8; ++i) p.g[i] = w[i] * (p.g[i] - s);
  __builtin_amdgcn_wave_barrier();
  return p;
}
static_assert(3 * 32 * MOE_MAX_TOPK <= 32 * tile_ld(kRbTile), "the pairs' staging lies in the tile");

// G of 32 tokens and experts e0 .. e0 + kE - 1 (32 or 64): requested (kRows: a first launch
// has written it) and put into the wavefront's tile.
template <int kE>
struct TileLoads {
  f32x4_t v[kE / 8];
};
template <bool kRows, int kE>
__device__ __forceinline__ TileLoads<kE> request_tile(const RouteBackDev& a, int64_t t0, int e0) {
  TileLoads<kE> r;
  constexpr int kLanes = kE / 4, kStep = 64 / kLanes;  // lanes per token, tokens per load
  if (kRows) {
    const MOE_GLOBAL char* base = (const MOE_GLOBAL char*)(a.g + t0 * a.Ep + e0);
    const uint32_t at = (lane_id() / kLanes) * a.Ep + lane_id() % kLanes * 4;
#pragma unroll
    for (int i = 0; i < kE / 8; ++i)
      r.v[i] = *(const MOE_GLOBAL f32x4_t*)(base + 4 * (at + kStep * i * (uint32_t)a.Ep));
  }
  return r;
}
template <bool kRows, int kE>
__device__ __forceinline__ void put_tile(float* tile, const TilePairs& p, const TileLoads<kE>& r, int e0) {
  const int lane = lane_id();
  constexpr int kLanes = kE / 4, kStep = 64 / kLanes, kLd = tile_ld(kE);
#pragma unroll
  for (int i = 0; i < kE / 8; ++i)
    *reinterpret_cast<f32x4_t*>(tile + (kStep * i + lane / kLanes) * kLd + lane % kLanes * 4) =
        kRows ? r.v[i] : f32x4_t{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_wave_barrier();
  if (!kRows) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = p.id[i] - e0;
      if (p.id[i] >= 0 && e >= 0 && e < kE) tile[(lane >> 1) * kLd + e] = p.g[i];
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// eight float32 values as kParts bf16 operands whose sum they are
template <int kParts>
__device__ __forceinline__ void split_parts(float (&v)[8], bf16x8_t (&part)[kParts]) {
#pragma unroll
  for (int s = 0; s < kParts; ++s) {
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      v[2 * i] -= __uint_as_float(q[i] << 16);
      v[2 * i + 1] -= __uint_as_float(q[i] & 0xFFFF0000u);
    }
    part[s] = as_bf16x8(q);
  }
}

// Eight elements of row r at column `col`, by a uniform base and a 32-bit offset
// (rows of up to 2^20 elements, at most 1024 of them).
__device__ __forceinline__ u32x4_t load_words(const uint16_t* base, uint32_t r, uint32_t d, uint32_t col) {
  return *(const MOE_GLOBAL u32x4_t*)((const MOE_GLOBAL char*)base + 2 * (r * d + col));
}

// Rows r0 .. r0 + 7 (clamped to the last) of a lane's eight columns ...
struct Block {
  uint32_t row[8][4];
};
__device__ __forceinline__ Block load_block(const uint16_t* base, int r0, int last, int d, int col) {
  Block b;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const u32x4_t v = load_words(base, r0 + r < last ? r0 + r : last, d, col);
#pragma unroll
    for (int i = 0; i < 4; ++i) b.row[r][i] = v[i];
  }
  return b;
}
// ... and column c of them, as eight k of an MFMA operand
__device__ __forceinline__ bf16x8_t column(const Block& b, int c) {
  u32x4_t v;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    v[p] = __builtin_amdgcn_perm(b.row[2 * p + 1][c >> 1], b.row[2 * p][c >> 1], (c & 1) ? 0x07060302u : 0x05040100u);
  return as_bf16x8(v);
}

// LDS of a workgroup: the wavefronts' tiles, then (dW) their sums
union alignas(16) RouteBackLds {
  float tile[kRbWaves][32 * tile_ld(kRbTile)];
  float sums[kRbWaves][16][kRbCols + 4];
};

// dx of a tile's 32 tokens in 128 columns: what is requested first ...
struct DxLoads {
  Block w;             // the first 32 experts
  TileLoads<kRbTile> g;  // the first 64
  uint32_t add[2][4][4];  // dx_add of the lane's results
};
template <bool kRows>
__device__ __forceinline__ DxLoads request_dx(const RouteBackDev& a, int64_t t0, int col) {
  const int kq = lane_id() >> 4;
  DxLoads r;
  r.g = request_tile<kRows, kRbTile>(a, t0, 0);
  r.w = load_block(a.w, 8 * kq, a.E - 1, a.d, col);
  const uint16_t* base = a.dx_add + t0 * a.d;
  const int last = (int)(a.T - 1 - t0 < 31 ? a.T - 1 - t0 : 31);
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * b + 4 * kq + q;
      u32x4_t v = {};
      if (a.dx_add) v = load_words(base, t < last ? t : last, a.d, col);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.add[b][q][i] = v[i];
    }
  return r;
}
// ... and the product, 32 experts a step.
template <bool kRows>
__device__ __forceinline__ void run_dx(const RouteBackDev& a, float* tile, const TilePairs& p, const DxLoads& r,
                                       int64_t t0, int col, bool stored) {
  const int lane = lane_id();
  const int n = lane & 15, kq = lane >> 4;
  f32x4_t acc[2][8];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Block next = r.w;
  TileLoads<kRbTile> tile_next = r.g;
  for (int e = 0; e < a.E; e += 32) {
    if (e % kRbTile == 0) {
      put_tile<kRows, kRbTile>(tile, p, tile_next, e);
      if (e + kRbTile < a.E) tile_next = request_tile<kRows, kRbTile>(a, t0, e + kRbTile);
    }
    const Block w = next;
    if (e + 32 < a.E) next = load_block(a.w, e + 32 + 8 * kq, a.E - 1, a.d, col);
    bf16x8_t gf[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float* row = tile + (16 * b + n) * tile_ld(kRbTile) + e % kRbTile + 8 * kq;
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(row), hi = *reinterpret_cast<const f32x4_t*>(row + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      split_parts<2>(v, gf[b]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x8_t wf = column(w, i);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[b][i] = mfma16x16x32(gf[b][s], wf, acc[b][i]);
    }
  }
  if (!stored) return;
  MOE_GLOBAL char* base = (MOE_GLOBAL char*)(a.dx + t0 * a.d);
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * b + 4 * kq + q;
      if (t0 + t >= a.T) continue;
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t add = r.add[b][q][i];
        o[i] = pack_bf16x2(acc[b][2 * i][q] + __uint_as_float(add << 16),
                           acc[b][2 * i + 1][q] + __uint_as_float(add & 0xFFFF0000u));
      }
      __builtin_nontemporal_store(
          o, (MOE_GLOBAL u32x4_t*)(base + 2 * ((uint32_t)t * (uint32_t)a.d + (uint32_t)col)));
    }
}

// dW: a workgroup sums 32 EB experts x 128 columns over its share of the tokens.  Its
// wavefronts take half of the experts each, for steps of 32 tokens of their own (four
// steps at a time); the four meet in LDS.
template <int EB, bool kRows>
__device__ __forceinline__ void route_dw(const RouteBackDev& a, int block, RouteBackLds& lds) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, kq = lane >> 4;
  const int half = wave & 1, group = wave >> 1;
  const int chunks = (a.d + kRbCols - 1) / kRbCols, tiles = (a.E + 32 * EB - 1) / (32 * EB);
  const int c0 = block % chunks * kRbCols;
  const int tile_e0 = block / chunks % tiles * 32 * EB, e0 = tile_e0 + half * 16 * EB;
  const int split = block / chunks / tiles;
  const int col = c0 + 8 * n < a.d ? c0 + 8 * n : 0;  // columns past the end: summed and not stored
  const int64_t steps = a.Tp / 32, stride = (int64_t)(kRbWaves / 2) * a.splits;
  float* tile = lds.tile[wave];
  f32x4_t acc[EB][8];
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int64_t st = split * (kRbWaves / 2) + group;
  auto load_x = [&](int64_t st) {
    const int64_t left = a.T - 1 - st * 32;
    return load_block(a.x + st * 32 * a.d, 8 * kq, (int)(left < 31 ? left : 31), a.d, col);
  };
  Block next;
  TileLoads<32> tile_next;
  if (st < steps) {
    tile_next = request_tile<kRows, 32>(a, st * 32, e0);
    next = load_x(st);
  }
  for (; st < steps; st += stride) {
    const int64_t t0 = st * 32;
    PairLoads r;
    if (!kRows) r = request_pairs(a, t0);
    const Block x = next;
    TilePairs p;
    if (!kRows) p = deal_pairs(a, r, t0, tile);
    put_tile<kRows, 32>(tile, p, tile_next, e0);
    if (st + stride < steps) {
      tile_next = request_tile<kRows, 32>(a, (st + stride) * 32, e0);
      next = load_x(st + stride);
    }
    bf16x8_t xf[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) xf[i] = column(x, i);
#pragma unroll
    for (int b = 0; b < EB; ++b) {
      if (e0 + 16 * b >= a.E) break;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = tile[(8 * kq + i) * tile_ld(32) + 16 * b + n];
      bf16x8_t gf[3];
      split_parts<3>(v, gf);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int s = 0; s < 3; ++s) acc[b][i] = mfma16x16x32(gf[s], xf[i], acc[b][i]);
    }
  }
  float* out = a.splits > 1 ? a.part + (int64_t)split * a.E * a.d : a.dw;
#pragma unroll
  for (int b = 0; b < EB; ++b) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float* p = &lds.sums[wave][4 * kq + q][8 * n];
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{acc[b][0][q], acc[b][1][q], acc[b][2][q], acc[b][3][q]};
      *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{acc[b][4][q], acc[b][5][q], acc[b][6][q], acc[b][7][q]};
    }
    __syncthreads();
    // both halves' 16 rows, four columns of two of them per thread
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      static_assert(kRbWaves * 64 == 16 * kRbCols / 4, "four columns of a row per thread");
      const int r = threadIdx.x / (kRbCols / 4), c = threadIdx.x % (kRbCols / 4) * 4;
      const int e = tile_e0 + h * 16 * EB + 16 * b + r;
      if (e < a.E && c0 + c < a.d) {
        f32x4_t v = *reinterpret_cast<const f32x4_t*>(&lds.sums[h][r][c]);
#pragma unroll
        for (int w = 1; w < kRbWaves / 2; ++w) v += *reinterpret_cast<const f32x4_t*>(&lds.sums[2 * w + h][r][c]);
        *reinterpret_cast<f32x4_t*>(out + (int64_t)e * a.d + c0 + c) = v;
      }
    }
  }
}

// dx alone: a wavefront computes 32 tokens x 128 columns.
template <bool kRows>
__device__ __forceinline__ void route_dx(const RouteBackDev& a, int block, RouteBackLds& lds) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int chunks = (a.d + kRbCols - 1) / kRbCols;
  const int at = block % chunks * kRbCols + 8 * (lane_id() & 15);
  const int64_t t0 = ((int64_t)(block / chunks) * kRbWaves + wave) * 32;
  if (t0 >= a.T) return;
  const int col = at < a.d ? at : 0;
  float* tile = lds.tile[wave];
  PairLoads r;
  if (!kRows) r = request_pairs(a, t0);
  const DxLoads dx = request_dx<kRows>(a, t0, col);
  TilePairs p;
  if (!kRows) p = deal_pairs(a, r, t0, tile);
  run_dx<kRows>(a, tile, p, dx, t0, col, at < a.d);
}

// Both products in one launch: the first dw_blocks workgroups sum dW, the others dx.
// (One workgroup that computes both from the same tiles ran slower, 36 against 23 us at
// T = 4096, d = 2048, E = 64: the registers of the two add up and spill.)
template <int EB, bool kRows>
__global__ __launch_bounds__(64 * kRbWaves) void k_route_products(RouteBackDev a, int dw_blocks) {
  __shared__ RouteBackLds lds;
  if ((int)blockIdx.x < dw_blocks)
    route_dw<EB, kRows>(a, blockIdx.x, lds);
  else
    route_dx<kRows>(a, blockIdx.x - dw_blocks, lds);
}

__global__ __launch_bounds__(256) void k_route_dw_sum(const float* part, int splits, int64_t count, float* dw) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(part + s * count + i);
  *reinterpret_cast<f32x4_t*>(dw + i) = v;
}

__global__ __launch_bounds__(256) void k_zero(float* p, int64_t count) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < count) p[i] = 0.f;
}

struct RouteBackPlan {
  int64_t Tp, g_bytes, part_bytes, total;
  int Ep, EB, splits;
};

static RouteBackPlan route_back_plan(int T, int d, int E) {
  RouteBackPlan p;
  p.Tp = ceil_div(T, 32) * 32;
  p.Ep = (int)ceil_div(E, kRbTile) * kRbTile;
  p.EB = E <= 32 ? 1 : 2;
  const int64_t tiles = ceil_div(d, kRbCols) * ceil_div(E, 32 * p.EB);
  const int64_t most = std::max<int64_t>(1, ceil_div(p.Tp / 32, kRbWaves / 2));
  // about 128 workgroups sum dW, so that those of dx run beside them (one workgroup fills a
  // CU) and few partial sums are left to add: T = 4096, d = 2048, E = 64 20.9 us, with 64
  // or 192 of them 29.4 or 24.4; T = 16384, E = 16 48.1, 78.4 or 49.2
  p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, ceil_div(128, tiles)));
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  p.g_bytes = up(p.Tp * p.Ep * 4);
  p.part_bytes = p.splits > 1 ? up((int64_t)p.splits * E * d * 4) : 0;
  p.total = p.g_bytes + p.part_bytes;
  return p;
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_route_backward_workspace_bytes(int T, int d, int E, int k) {
  if (T < 0 || d <= 0 || E <= 0 || k <= 0) return -1;
  return route_back_plan(T, d, E).total;
}

extern "C" int moe_route_backward(const moe_route_backward_args* a, void* stream) {
  clear_error();
  MOE_CHECK_ARG(a != nullptr, MOE_ERR_INVALID_ARG, "moe_route_backward: args is NULL");
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0 && a->E > 0 && a->k > 0, MOE_ERR_INVALID_ARG,
                "moe_route_backward: bad sizes T=%d d=%d E=%d k=%d", a->T, a->d, a->E, a->k);
  MOE_CHECK_ARG(a->E <= MOE_MAX_EXPERTS && a->k <= MOE_MAX_TOPK && a->k <= a->E && a->d % 8 == 0 &&
                    a->d <= (1 << 20) && a->T <= (1 << 24),
                MOE_ERR_UNSUPPORTED_SHAPE,
                "moe_route_backward: unsupported E=%d k=%d d=%d T=%d (E <= 1024, k <= min(E,16), d %% 8 == 0, "
                "d <= 2^20, T <= 2^24)",
                a->E, a->k, a->d, a->T);
  MOE_CHECK_ARG(((uintptr_t)a->dw_router % 16) == 0, MOE_ERR_INVALID_ARG, "moe_route_backward: misaligned dw_router");
  hipStream_t s = (hipStream_t)stream;
  if (a->T == 0) {
    if (!a->dw_router) return MOE_OK;
    const int64_t count = (int64_t)a->E * a->d;
    hipLaunchKernelGGL(k_zero, dim3((unsigned)ceil_div(count, 256)), dim3(256), 0, s, a->dw_router, count);
    return check_launch("moe_route_backward");
  }
  MOE_CHECK_ARG(a->topk_ids && a->topk_weights && a->dweights && (a->logits || a->renormalize) && (a->dx || a->dw_router),
                MOE_ERR_INVALID_ARG, "moe_route_backward: null pointer");
  MOE_CHECK_ARG((!a->dx || a->w_router) && (!a->dw_router || a->x), MOE_ERR_INVALID_ARG,
                "moe_route_backward: dx needs w_router, dw_router needs x");
  MOE_CHECK_ARG(((uintptr_t)a->x % 16) == 0 && ((uintptr_t)a->w_router % 16) == 0 && ((uintptr_t)a->dx % 16) == 0 &&
                    ((uintptr_t)a->dx_add % 16) == 0,
                MOE_ERR_INVALID_ARG, "moe_route_backward: x, w_router, dx and dx_add must be 16-byte aligned");
  for (const void* p : {(const void*)a->logits, (const void*)a->topk_ids, (const void*)a->topk_weights,
                        (const void*)a->dweights, (const void*)a->dlogits})
    MOE_CHECK_ARG(((uintptr_t)p % 4) == 0, MOE_ERR_INVALID_ARG, "moe_route_backward: misaligned input");
  const RouteBackPlan p = route_back_plan(a->T, a->d, a->E);
  MOE_CHECK_ARG(a->workspace && ((uintptr_t)a->workspace % 256) == 0 && a->workspace_bytes >= p.total,
                MOE_ERR_WORKSPACE, "moe_route_backward: workspace NULL, misaligned or %lld bytes < %lld needed",
                (long long)a->workspace_bytes, (long long)p.total);
  RouteBackDev v;
  v.x = a->x;
  v.w = a->w_router;
  v.T = a->T;
  v.d = a->d;
  v.E = a->E;
  v.k = a->k;
  v.renormalize = a->renormalize;
  v.Tp = p.Tp;
  v.Ep = p.Ep;
  v.logits = a->logits;
  v.ids = a->topk_ids;
  v.weights = a->topk_weights;
  v.dweights = a->dweights;
  v.dlogits = a->dlogits;
  v.dx_add = a->dx_add;
  v.dx = a->dx;
  v.dw = a->dw_router;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  v.g = a->renormalize && !a->dlogits ? nullptr : reinterpret_cast<float*>(ws);
  v.part = reinterpret_cast<float*>(ws + p.g_bytes);
  v.splits = p.splits;
  timing_begin(K_ROUTE_BWD, s);
  if (v.g) {
    const dim3 grid((unsigned)(p.Tp / 4));
    if (p.Ep <= 64)
      hipLaunchKernelGGL(k_route_dlogits<1>, grid, dim3(256), 0, s, v);
    else if (p.Ep <= 256)
      hipLaunchKernelGGL(k_route_dlogits<4>, grid, dim3(256), 0, s, v);
    else
      hipLaunchKernelGGL(k_route_dlogits<16>, grid, dim3(256), 0, s, v);
  }
  const int64_t chunks = ceil_div(a->d, kRbCols);
  const int64_t dw_blocks = a->dw_router ? chunks * ceil_div(a->E, 32 * p.EB) * p.splits : 0;
  const int64_t dx_blocks = a->dx ? chunks * ceil_div(a->T, 32 * kRbWaves) : 0;
  auto products = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(dw_blocks + dx_blocks)), dim3(64 * kRbWaves), 0, s, v, (int)dw_blocks);
  };
  if (p.EB == 1)
    v.g ? products(k_route_products<1, true>) : products(k_route_products<1, false>);
  else
    v.g ? products(k_route_products<2, true>) : products(k_route_products<2, false>);
  if (a->dw_router && p.splits > 1) {
    const int64_t count = (int64_t)a->E * a->d;
    hipLaunchKernelGGL(k_route_dw_sum, dim3((unsigned)ceil_div(count, 1024)), dim3(256), 0, s, v.part, p.splits, count,
                       a->dw_router);
  }
  timing_end(K_ROUTE_BWD, s);
  return check_launch("moe_route_backward");
}

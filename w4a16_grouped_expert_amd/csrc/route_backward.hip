// moe_route_backward: from the gradient of the routing weights to those of the router's
// input and weight (ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient
// W4A16 Inference", Abstract: BF16 router, unchanged top-k).
//
// With G [T][E] the gradient of the logits, dx = G W (+ dx_add) and dW = G^T x.  W and x
// are bf16 as they are; G is split into bf16 parts whose sum is G to 2^-18 (two parts,
// for dx, which is rounded to bf16) or 2^-27 (three parts, for the float32 dW), so both
// products run on the bf16 matrix cores with float32 sums.
//
// A first launch computes G and writes its parts as the 16x16x32 MFMA takes its first
// operand, eight consecutive k per lane: for dx [E/8][T][8], for dW [T/8][E][8].  The
// products load them without further work (splitting G in every wavefront that needs it:
// 31 in place of 24 us at T = 1021, d = 4096, E = 257).  With few experts and k values per
// token the products build G from the pairs themselves and save the launch.
//
// The second operand's k runs over the rows of a row-major bf16 matrix (W over e, x over
// t): a thread loads eight rows of 16 bytes (eight columns), and v_perm pairs the rows,
// which transposes the 8 x 8 block in registers.  MFMA i of eight has column 8n + i as its
// column n, so a lane ends with eight consecutive columns of the result.  W, which every
// wavefront of a workgroup of dx needs, goes through LDS; the blocks of x stay in the
// registers of their wavefront, without a barrier behind which the next loads would wait
// (x through LDS too: dW alone 11.3 to 12.5 us at T = 4096, d = 2048, E = 64).
//
// Measured: T = 4096, d = 2048, E = 64, k = 8 from the pairs 16.4 us and 3.9 for the sum of
// dW's parts (52 MB with dx_add); T = 1021, d = 4096, E = 257 5.6 us for G, 19.7 for the
// products.  A step of 32 rows loads 14 KB per wavefront of dW (x and three parts of G) for
// 48 MFMA.  From the pairs a wavefront of dW has few such steps (four at T = 4096) and waits in each
// for its pairs, which are not requested early.  With many experts the workgroups spread
// unevenly (see route_back_plan).
#include "rows.hpp"

namespace moe {

constexpr int kRbCols = 128;   // columns of d per wavefront
constexpr int kRbWaves = 4;    // wavefronts per workgroup of the products
constexpr int kRbStep = 32;    // rows of one MFMA
// With the softmax over the selected experts, no loss on the logits and at most this many
// experts, the wavefronts of the products build G from the pairs themselves, in tiles of
// 32 tokens in LDS: no first launch (E = 64, d = 2048: T = 64 5.8 us in place of 8.1,
// at T = 4096 the same either way).  A tile of more experts would be built once per 64.
constexpr int kPairExperts = 64;
constexpr int kTileFloats = 32 * (kPairExperts + 4);
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
  u32x4_t* g_dx;  // [2 parts][Ep / 8][Tp] eight experts of a token; null: dx not wanted
  u32x4_t* g_dw;  // [3 parts][Tp / 8][Ep] eight tokens of an expert; null: dw not wanted
  float* part;    // [splits][E][d] where splits > 1
  int splits;
};

// eight float32 values as kParts bf16 operands whose sum they are
template <int kParts>
__device__ __forceinline__ void split_parts(float (&v)[8], u32x4_t (&part)[kParts]) {
#pragma unroll
  for (int s = 0; s < kParts; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      part[s][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      v[2 * i] -= __uint_as_float(part[s][i] << 16);
      v[2 * i + 1] -= __uint_as_float(part[s][i] & 0xFFFF0000u);
    }
  }
}

// the largest of 64 lanes' values, in each of them
template <int kCtrl>
__device__ __forceinline__ float max_dpp(float v) {
  const int b = __float_as_int(v);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, kCtrl, 0xF, 0xF, false)));
}
__device__ __forceinline__ float lane_max(float v) {
  v = max_dpp<0xB1>(v);  // the steps of lane_sum
  v = max_dpp<0x4E>(v);
  v = max_dpp<0x141>(v);
  v = max_dpp<0x140>(v);
  uint32_t b = __float_as_uint(v);
  u32x2_t s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(b, b, false, false));
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  b = __float_as_uint(v);
  s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// G of eight tokens, a wavefront each, its E <= 64 kEL logits (read once) in the lanes'
// registers; through LDS into both operand layouts.  Rows past T and columns past E are
// zero.
template <int kEL>
__global__ __launch_bounds__(512) void k_route_g(RouteBackDev a) {
  constexpr int kLd = 64 * kEL + 4;  // (rows stay 16-byte aligned)
  __shared__ alignas(16) float tile[8][kLd];
  const int lane = lane_id();
  const int64_t t0 = (int64_t)blockIdx.x * 8, t = t0 + (threadIdx.x >> 6);
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
      top = lane_max(top);
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
    for (int i = 0; i < kEL; ++i) v[i] = lane + 64 * i < a.E ? v[i] + add[i] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kEL; ++i) tile[threadIdx.x >> 6][lane + 64 * i] = v[i];
  __syncthreads();
  if (a.g_dw) {
    u32x4_t* out = a.g_dw + (int64_t)blockIdx.x * a.Ep;
    for (int e = threadIdx.x; e < a.Ep; e += 512) {
      float q[8];
      u32x4_t part[3];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = tile[i][e];
      split_parts<3>(q, part);
#pragma unroll
      for (int s = 0; s < 3; ++s) out[s * (a.Tp / 8) * a.Ep + e] = part[s];
    }
  }
  if (a.g_dx) {
    u32x4_t* out = a.g_dx + t0 + (threadIdx.x & 7);
    for (int o = threadIdx.x >> 3; o < a.Ep / 8; o += 64) {
      const f32x4_t* row = reinterpret_cast<const f32x4_t*>(&tile[threadIdx.x & 7][8 * o]);
      const f32x4_t lo = row[0], hi = row[1];
      float q[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      u32x4_t part[2];
      split_parts<2>(q, part);
#pragma unroll
      for (int s = 0; s < 2; ++s) out[((int64_t)s * (a.Ep / 8) + o) * a.Tp] = part[s];
    }
  }
}

// G from the pairs.  What a wavefront needs to build tiles of 32 tokens: two lanes per
// token, each with every other of its pairs.  The tokens' pairs lie one after the other:
// they are loaded in that order (whole cache lines) and dealt out through the wavefront's
// tile.
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
static_assert(3 * 32 * MOE_MAX_TOPK <= kTileFloats, "the pairs' staging lies in the tile");

// the experts e0 .. e0 + kE - 1 (32 or 64) of the tokens into the wavefront's tile
constexpr int tile_ld(int kE) { return kE + 4; }  // floats per token: rows stay 16-byte aligned
template <int kE>
__device__ __forceinline__ void put_tile(float* tile, const TilePairs& p, int e0) {
  const int lane = lane_id();
  constexpr int kLanes = kE / 4, kStep = 64 / kLanes, kLd = tile_ld(kE);
  static_assert(32 * kLd <= kTileFloats, "a tile");
#pragma unroll
  for (int i = 0; i < kE / 8; ++i)
    *reinterpret_cast<f32x4_t*>(tile + (kStep * i + lane / kLanes) * kLd + lane % kLanes * 4) =
        f32x4_t{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = p.id[i] - e0;
    if (p.id[i] >= 0 && e >= 0 && e < kE) tile[(lane >> 1) * kLd + e] = p.g[i];
  }
  __builtin_amdgcn_wave_barrier();
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

// G of two groups of 16 tokens or experts, as first operands.
template <int kTiles, int kParts>
struct Operands {
  u32x4_t v[kTiles][kParts];
};
// acc += G (the rows whose columns `column` gives)
template <int kTiles, int kParts, typename F>
__device__ __forceinline__ void multiply(const Operands<kTiles, kParts>& g, f32x4_t (&acc)[kTiles][8], F column) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bf16x8_t c = column(i);
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int m = 0; m < kTiles; ++m) acc[m][i] = mfma16x16x32(as_bf16x8(g.v[m][p]), c, acc[m][i]);
  }
}

// dx: 32 tokens x 128 columns per wavefront.  128 rows of W at a time are in LDS, a thread
// transposes one 8 x 8 block of them: [row / 8][i][n] eight rows of column 8n + i.
template <bool kPairs>
__device__ __forceinline__ void route_dx(const RouteBackDev& a, int block, u32x4_t* lds, float* tile) {
  constexpr int kRows = 32 * kRbWaves, kSteps = kRows / kRbStep;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, kq = lane >> 4;
  const int chunks = (a.d + kRbCols - 1) / kRbCols;
  const int at = block % chunks * kRbCols + 8 * n;
  const int col = at < a.d ? at : 0;  // columns past the end: computed and not stored
  const int64_t tw = ((int64_t)(block / chunks) * kRbWaves + wave) * 32;
  const bool live = tw < a.T;
  const int64_t t0 = live ? tw : 0;
  const int steps = (a.E + kRbStep - 1) / kRbStep;
  const uint32_t lane_at = 16u * ((uint32_t)kq * (uint32_t)a.Tp + n);
  auto load_g = [&](int st) {
    Operands<2, 2> r;
    if (kPairs) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float* row = tile + (16 * m + n) * tile_ld(kPairExperts) + st % 2 * kRbStep + 8 * kq;
        const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(row), hi = *reinterpret_cast<const f32x4_t*>(row + 4);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        split_parts<2>(v, r.v[m]);
      }
      return r;
    }
    st = st < steps ? st : steps - 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const u32x4_t* base = uniform_ptr(a.g_dx + ((int64_t)s * (a.Ep / 8) + 4 * st) * a.Tp + t0);
#pragma unroll
      for (int m = 0; m < 2; ++m) r.v[m][s] = *(const MOE_GLOBAL u32x4_t*)((const MOE_GLOBAL char*)(base + 16 * m) + lane_at);
    }
    return r;
  };
  const int o = (int)threadIdx.x / 16;  // (the thread's block: rows 8 o .., the lane's columns)
  auto put = [&](const Block& b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[(o * 8 + i) * 16 + n] = __builtin_bit_cast(u32x4_t, column(b, i));
  };
  PairLoads r;
  if (kPairs) r = request_pairs(a, t0);
  Block w = load_block(a.w, 8 * o, a.E - 1, a.d, col);
  if (kPairs) put_tile<kPairExperts>(tile, deal_pairs(a, r, t0, tile), 0);
  Operands<2, 2> g = load_g(0);
  f32x4_t acc[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto run = [&](int first, int end) {
#pragma unroll 1
    for (int st = first; st < end; ++st) {
      const Operands<2, 2> next = load_g(st + 1);
      multiply(g, acc, [&](int i) { return as_bf16x8(lds[(((st - first) * (kRbStep / 8) + kq) * 8 + i) * 16 + n]); });
      g = next;
    }
  };
  int e0 = 0;
#pragma unroll 1
  for (; e0 + kRows < a.E; e0 += kRows) {
    put(w);
    __syncthreads();
    w = load_block(a.w, e0 + kRows + 8 * o, a.E - 1, a.d, col);
    run(e0 / kRbStep, e0 / kRbStep + kSteps);
    __syncthreads();
  }
  put(w);
  __syncthreads();
  // dx_add of the results (or a row of W that becomes zero) beside the last steps
  const int last = (int)(a.T - 1 - t0 < 31 ? a.T - 1 - t0 : 31);
  const uint16_t* add_base = a.dx_add ? a.dx_add + t0 * a.d : a.w;
  const uint32_t on = a.dx_add ? ~0u : 0u;
  u32x4_t add[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * m + 4 * kq + q;
      add[m][q] = load_words(add_base, (t < last ? t : last) & on, a.d, col);
    }
  run(e0 / kRbStep, steps);
  if (!live || at >= a.d) return;
  MOE_GLOBAL char* base = (MOE_GLOBAL char*)(a.dx + t0 * a.d);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * m + 4 * kq + q;
      if (t0 + t >= a.T) continue;
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = add[m][q][i] & on;
        o[i] = pack_bf16x2(acc[m][2 * i][q] + __uint_as_float(v << 16),
                           acc[m][2 * i + 1][q] + __uint_as_float(v & 0xFFFF0000u));
      }
      __builtin_nontemporal_store(o, (MOE_GLOBAL u32x4_t*)(base + 2 * ((uint32_t)t * (uint32_t)a.d + (uint32_t)col)));
    }
}

// dW: a workgroup sums 16 EB experts x 128 columns over its share of the tokens.  Its
// wavefronts take every fourth step of 32 tokens and meet in LDS.
template <int EB, bool kPairs>
__device__ __forceinline__ void route_dw(const RouteBackDev& a, int block, f32x4_t* lds, float* tile) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, kq = lane >> 4;
  const int chunks = (a.d + kRbCols - 1) / kRbCols, tiles = (a.E + 16 * EB - 1) / (16 * EB);
  const int c0 = block % chunks * kRbCols;
  const int e0 = block / chunks % tiles * 16 * EB;
  const int split = block / chunks / tiles;
  const int col = c0 + 8 * n < a.d ? c0 + 8 * n : 0;  // columns past the end: summed and not stored
  const int64_t steps = a.Tp / kRbStep, stride = (int64_t)kRbWaves * a.splits;
  const uint32_t lane_at = 16u * ((uint32_t)kq * (uint32_t)a.Ep + n);
  auto load_g = [&](int64_t st) {
    Operands<EB, 3> r;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const u32x4_t* base = uniform_ptr(a.g_dw + (s * (a.Tp / 8) + 4 * st) * a.Ep + e0);
#pragma unroll
      for (int b = 0; b < EB; ++b) r.v[b][s] = *(const MOE_GLOBAL u32x4_t*)((const MOE_GLOBAL char*)(base + 16 * b) + lane_at);
    }
    return r;
  };
  auto load_x = [&](int64_t st) {
    const int64_t left = a.T - 1 - st * kRbStep;
    return load_block(a.x + st * kRbStep * a.d, 8 * kq, (int)(left < 31 ? left : 31), a.d, col);
  };
  f32x4_t acc[EB][8];
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int64_t st = split * kRbWaves + wave;
  if (kPairs && st < steps) {
    Block x = load_x(st);
#pragma unroll 1
    for (; st < steps; st += stride) {
      const PairLoads r = request_pairs(a, st * kRbStep);
      const Block x_next = load_x(st + stride < steps ? st + stride : st);
      put_tile<32>(tile, deal_pairs(a, r, st * kRbStep, tile), e0);
      Operands<EB, 3> g;
#pragma unroll
      for (int b = 0; b < EB; ++b) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = tile[(8 * kq + i) * tile_ld(32) + 16 * b + n];
        split_parts<3>(v, g.v[b]);
      }
      multiply(g, acc, [&](int i) { return column(x, i); });
      x = x_next;
    }
  }
  if (!kPairs && st < steps) {
    Operands<EB, 3> g = load_g(st);
    Block x = load_x(st);
#pragma unroll 1
    for (; st + stride < steps; st += stride) {
      const Operands<EB, 3> g_next = load_g(st + stride);
      const Block x_next = load_x(st + stride);
      multiply(g, acc, [&](int i) { return column(x, i); });
      g = g_next;
      x = x_next;
    }
    multiply(g, acc, [&](int i) { return column(x, i); });
  }
  // [wavefront][j][lane], vector j of 16 bytes: four columns 8n + 4 (j & 1) of expert
  // 4 kq + j / 2.  Each wavefront adds two of the vectors, over the wavefronts in order.
  float* out = a.splits > 1 ? a.part + (int64_t)split * a.E * a.d : a.dw;
#pragma unroll
  for (int b = 0; b < EB; ++b) {
    if (b) __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      lds[(wave * 8 + j) * 64 + lane] = f32x4_t{acc[b][4 * (j & 1)][j >> 1], acc[b][4 * (j & 1) + 1][j >> 1],
                                                acc[b][4 * (j & 1) + 2][j >> 1], acc[b][4 * (j & 1) + 3][j >> 1]};
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 8 / kRbWaves; ++m) {
      const int j = wave * (8 / kRbWaves) + m, e = e0 + 16 * b + 4 * kq + (j >> 1), c = c0 + 8 * n + 4 * (j & 1);
      f32x4_t v = lds[j * 64 + lane];
#pragma unroll
      for (int q = 1; q < kRbWaves; ++q) v += lds[(q * 8 + j) * 64 + lane];
      if (e < a.E && c < a.d) *reinterpret_cast<f32x4_t*>(out + (int64_t)e * a.d + c) = v;
    }
  }
}

// Both products in one launch: the first dw_blocks workgroups sum dW, the others dx.  (Three
// workgroups per CU leave 168 registers: with EB = 2 and G read three of them are spilled.)
template <int EB, bool kPairs>
__global__ __launch_bounds__(64 * kRbWaves, kPairs ? 2 : 3) void k_route_products(RouteBackDev a, int dw_blocks) {
  // dW: the wavefronts' sums; dx: 128 rows of W
  __shared__ u32x4_t lds[kRbWaves * 8 * 64];
  __shared__ alignas(16) float tiles[kPairs ? kRbWaves : 1][kPairs ? kTileFloats : 1];
  float* tile = tiles[kPairs ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0];
  if ((int)blockIdx.x < dw_blocks)
    route_dw<EB, kPairs>(a, blockIdx.x, reinterpret_cast<f32x4_t*>(lds), tile);
  else
    route_dx<kPairs>(a, blockIdx.x - dw_blocks, lds, tile);
}

// dW from its parts, in order: 4 us for 8 parts of 64 x 2048, a launch and their loads.
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
  int64_t Tp, g_dx_bytes, g_dw_bytes, part_bytes, total;
  int Ep, EB, splits;
};

// what the call takes, of sizes that are positive (T: not negative)
static bool route_back_takes(int T, int d, int E, int k) {
  return E <= MOE_MAX_EXPERTS && k <= MOE_MAX_TOPK && k <= E && d % 8 == 0 && d <= (1 << 20) && T <= (1 << 24);
}

static RouteBackPlan route_back_plan(int T, int d, int E) {
  RouteBackPlan p;
  p.Tp = ceil_div(T, kRbStep) * kRbStep;
  p.Ep = (int)ceil_div(E, 64) * 64;
  p.EB = E <= 16 ? 1 : 2;
  const int64_t tiles = ceil_div(d, kRbCols) * ceil_div(E, 16 * p.EB);
  const int64_t most = std::max<int64_t>(1, ceil_div(p.Tp / kRbStep, kRbWaves));
  // About 256 workgroups sum dW beside those of dx: at T = 4096, d = 2048, E = 64, the one size
  // tried, 192 or 384 of them take 8 % longer.  Those of dx are not counted, nor a last tile of
  // few experts: T = 1021, d = 4096, E = 257 has 288 and 256 workgroups for 256 CUs, 32 of them for
  // one expert.
  p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, ceil_div(256, tiles)));
  p.g_dx_bytes = 2 * p.Tp * p.Ep * 2;  // (multiples of 4096)
  p.g_dw_bytes = 3 * p.Tp * p.Ep * 2;
  p.part_bytes = p.splits > 1 ? (int64_t)p.splits * E * d * 4 : 0;
  p.total = std::max<int64_t>(256, p.g_dx_bytes + p.g_dw_bytes + p.part_bytes);
  return p;
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_route_backward_workspace_bytes(int T, int d, int E, int k) {
  if (T < 0 || d <= 0 || E <= 0 || k <= 0 || !route_back_takes(T, d, E, k)) return -1;
  return route_back_plan(T, d, E).total;
}

extern "C" int moe_route_backward(const moe_route_backward_args* a, void* stream) {
  clear_error();
  MOE_CHECK_ARG(a != nullptr, MOE_ERR_INVALID_ARG, "moe_route_backward: args is NULL");
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0 && a->E > 0 && a->k > 0, MOE_ERR_INVALID_ARG,
                "moe_route_backward: bad sizes T=%d d=%d E=%d k=%d", a->T, a->d, a->E, a->k);
  MOE_CHECK_ARG(route_back_takes(a->T, a->d, a->E, a->k), MOE_ERR_UNSUPPORTED_SHAPE,
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
  v.g_dx = a->dx ? reinterpret_cast<u32x4_t*>(ws) : nullptr;
  v.g_dw = a->dw_router ? reinterpret_cast<u32x4_t*>(ws + p.g_dx_bytes) : nullptr;
  v.part = reinterpret_cast<float*>(ws + p.g_dx_bytes + p.g_dw_bytes);
  v.splits = p.splits;
  const bool pairs = a->renormalize && !a->dlogits && a->E <= kPairExperts;
  timing_begin(K_ROUTE_BWD, s);
  if (!pairs) {
    auto write_g = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)(p.Tp / 8)), dim3(512), 0, s, v); };
    if (p.Ep <= 64)
      write_g(k_route_g<1>);
    else if (p.Ep <= 128)
      write_g(k_route_g<2>);
    else if (p.Ep <= 256)
      write_g(k_route_g<4>);
    else if (p.Ep <= 512)
      write_g(k_route_g<8>);
    else
      write_g(k_route_g<16>);
  }
  const int64_t chunks = ceil_div(a->d, kRbCols);
  const int64_t dw_blocks = a->dw_router ? chunks * ceil_div(a->E, 16 * p.EB) * p.splits : 0;
  const int64_t dx_blocks = a->dx ? chunks * ceil_div(a->T, 32 * kRbWaves) : 0;
  auto products = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(dw_blocks + dx_blocks)), dim3(64 * kRbWaves), 0, s, v, (int)dw_blocks);
  };
  if (p.EB == 1)
    pairs ? products(k_route_products<1, true>) : products(k_route_products<1, false>);
  else
    pairs ? products(k_route_products<2, true>) : products(k_route_products<2, false>);
  if (a->dw_router && p.splits > 1) {
    const int64_t count = (int64_t)a->E * a->d;
    hipLaunchKernelGGL(k_route_dw_sum, dim3((unsigned)ceil_div(count, 1024)), dim3(256), 0, s, v.part, p.splits, count,
                       a->dw_router);
  }
  timing_end(K_ROUTE_BWD, s);
  return check_launch("moe_route_backward");
}

// Gated feed-forward blocks with 16-bit weights, and their gradient: the experts of a
// training step over rows sorted by expert, or one dense block over all rows (ExactMoE, page
// "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference", Abstract: every selected
// expert runs through fused grouped kernels; it names no activation and no training).
//
//   g = x Wg^T, u = x Wu^T, h = drop(act(g) u), y = h Wd^T
//   dh = drop(dy Wd), dg = dh u act'(g), du = dh act(g)
//   dx = [dg, du] W13, dW13 = [dg, du]^T x, dWd = dy^T h
//
// Six products on the matrix cores (tile_product.hpp), each one launch over all experts:
//   gate/up   A = rows (k = d), B = W13, gate and up rows of the same 128 columns in one tile:
//             activation, product and dropout are applied to the float32 sums
//   down      A = h, B = Wd
//   dh        A = dy, B = Wd with n contiguous; dg and du are formed from the float32 sums
//   dx        A = [dg, du], B = W13 with n contiguous
//   dW13, dWd A and B with the rows as k, per expert
// h, dg and du are rounded to the tensors' type once, as the operands of the next product: a
// bf16 output is then off by 0.0024 in the 2-norm where one rounding alone makes it 0.0017.  In fp16
// that is a range as well: beyond 65504 they are infinite, below 2^-25 zero.
//
// What bounds them, at 1.2 to 1.45 PFLOP/s that large library products reach here: one dense
// block (R = 4096, d = 2048, I = 8192, gradient) runs at 1.12 PFLOP/s; per unit of 64 k a tile of
// 256 x 256 needs its matrix cores for 2048 cycles, its LDS for as many (192 KB read, 64 KB
// written) and its DMA for half of them, and they do not overlap fully (matrix cores busy for 0.57
// to 0.64 of the weights' gradients' time).  Over 64 experts of some 512 rows (d = 2048, I = 1024)
// 815 TFLOP/s forward and 755 backward, matrix cores busy for 0.27 to 0.40: each workgroup has an
// equal number of tiles, not equal work (gate/up: six at most where the mean by products is 4.4;
// the CUs have a wavefront for 0.77 of its time), the last tile of an expert is partly empty (1.08
// times the products), the weights are read from memory for two tiles of rows each, and 2 bytes
// per weight of gradients are stored behind eight units of products.  dg and du: g and u are
// requested behind a tile's last product (matrix cores 0.34 of the time dense, 0.27 grouped).
#include <cmath>

#include "philox.hpp"
#include "tile_product.hpp"

namespace moe {

enum ProductKind { kGateUp, kDown, kGateBack, kRowsBack, kWeightBack };

constexpr int kXcds = 8;

struct ProductDev {
  const char* a;
  const char* b;
  int64_t b_expert;   // bytes between two experts' weights
  int lda, ldb;       // elements
  int M, N, K;        // kWeightBack: K by expert; else M by expert
  int R, E;
  const int32_t* offsets;  // or NULL: one expert, all rows
  char* out;          // kGateUp: h; kGateBack: [dg, du]
  int ldo;
  char* gu;           // kGateUp: written unless NULL; kGateBack: read
  int ldgu;
  int activation;
  DropDev drop;
};

// Rows of expert e, clamped to the R that are there.
__device__ __forceinline__ void expert_rows(const ProductDev& p, int e, int& row0, int& count) {
  if (!p.offsets) {
    row0 = 0;
    count = p.R;
    return;
  }
  row0 = min(max(p.offsets[e], 0), p.R);
  count = max(min(p.offsets[e + 1], p.R) - row0, 0);
}

// The activation and its derivative, both by one logistic function (gelu in its tanh form is
// g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)); hardware exp and reciprocal, a
// few units in the last place of float32 before a rounding to 16 bits.
__device__ __forceinline__ float activate(int activation, float g, float& slope) {
  float s = g, ds = 1.f;
  if (activation == MOE_ACT_GELU) {
    const float c = fminf(fmaxf(g, -30.f), 30.f), c2 = c * c;  // saturated beyond
    s = 1.5957691216f * c * fmaf(0.044715f, c2, 1.f);
    ds = 1.5957691216f * fmaf(0.134145f, c2, 1.f);
  }
  const float p = __builtin_amdgcn_rcpf(1.f + __expf(-s));
  const float a = g * p;
  slope = fmaf(a * (1.f - p), ds, p);
  return a;
}

template <typename S>
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  return pack<S>(v).w[0];
}

// The lane's number as a value that the compiler does not see through: what follows from it is
// computed where it is used, in place of registers held through the products.
__device__ __forceinline__ int fresh_lane() {
  int l = lane_id();
  asm volatile("" : "+v"(l));
  return l;
}

// One tile of a product.
struct Tile {
  int e, row0, m0, n0, m_left, K;
};

// Persistent workgroups, each with its tiles in turn.  All loads are issued kUnits - 1 units ahead
// of the products by a cursor of its own, which runs into the next tiles while this one ends.
//
// Tile shapes: wavefronts, those of them in m, blocks of 16 rows and columns of each, units of the
// ring and workgroups per CU.
template <int waves, int wm, int mi, int ni, int units, int per_cu>
struct Shape {
  static constexpr int kWaves = waves, kWM = wm, kMI = mi, kNI = ni, kUnits = units, kPerCu = per_cu;
  static constexpr int kTileM = wm * mi * 16, kTileN = waves / wm * ni * 16;
};
typedef Shape<8, 2, 8, 4, 2, 1> Shape256;   // 256 x 256
typedef Shape<8, 2, 4, 4, 3, 1> Shape128;   // 128 x 256
typedef Shape<8, 2, 2, 4, 3, 1> Shape64;    // 64 x 256
typedef Shape<4, 2, 4, 4, 2, 2> ShapeHalf;  // 128 x 128, two workgroups per CU

template <typename S, int kKind, typename Sh>
__global__ __launch_bounds__(64 * Sh::kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_product(ProductDev p) {
  constexpr int kWaves = Sh::kWaves, kWM = Sh::kWM, kMI = Sh::kMI, kNI = Sh::kNI, kUnits = Sh::kUnits;
  constexpr int kTileM = Sh::kTileM, kTileN = Sh::kTileN;
  constexpr bool kDual = kKind == kGateUp;
  constexpr bool kAMContig = kKind == kWeightBack;
  constexpr bool kBMContig = kKind >= kGateBack;
  constexpr int kCols = kDual ? kTileN / 2 : kTileN;
  constexpr int kHalf = kDual ? kNI / 2 : kNI;  // blocks of a wavefront within a tensor
  typedef Stager<kTileM, kWaves, kAMContig> StageA;
  typedef Stager<kTileN, kWaves, kBMContig, kDual> StageB;
  constexpr int kStage = StageA::kBytes + StageB::kBytes;
  constexpr int kIssues = StageA::kIssues + StageB::kIssues;
  constexpr int kPending = (kUnits - 2) * kIssues;
  constexpr int kAhead = kUnits + 1;  // the tiles that the cursor may be ahead, and this one
  // stores of a tile's epilogue per wavefront (without those of g and u, which may be missing)
  constexpr int kPairs = kNI / 2;  // pairs of column blocks
  constexpr int kStores = (kKind == kGateUp ? 1 : kKind == kGateBack ? 2 * kPairs : kPairs) * kMI;
  static_assert(kPending + kStores < 64, "the counter's six bits");
  __shared__ __attribute__((aligned(1024))) char s_stage[kUnits * kStage];
  __shared__ int s_first[kKind == kWeightBack ? 1 : MOE_MAX_EXPERTS + 1];  // first m tile of each expert
  __shared__ Tile s_tile[kWaves][kAhead];  // each wavefront's own copy of the tiles ahead

  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % kWM, wn = wave / kWM;
  const int NT = (p.N + kCols - 1) / kCols;

  // ---- the tiles: m tiles of each expert, one expert behind the other.  Each XCD takes a
  // contiguous run of them, so that those that share operands meet in its L2, of an equal share of
  // the work: for the weights' gradients, whose experts have unequal K, units and the store.
  int m_tiles;
  const int xcd = blockIdx.x % kXcds, per_xcd = gridDim.x / kXcds;
  int from_tile, last_tile;
  if constexpr (kKind == kWeightBack) {
    m_tiles = (p.M + kTileM - 1) / kTileM;
    const int per_expert = m_tiles * NT;
    // (a tile's store costs about as much as kStoreUnits units)
    constexpr int kStoreUnits = 4;
    auto cost_of = [&](int e) {
      int row0, count = 0;
      if (e < p.E) expert_rows(p, e, row0, count);
      return e < p.E ? (count + kUnitK - 1) / kUnitK + kStoreUnits : 0;
    };
    int whole = 0;  // cost of one tile of every expert: below 2^24 / 64 + 5 E
    for (int base = 0; base < p.E; base += 64) whole += cost_of(base + lane);
    for (int off = 32; off; off >>= 1) whole += __shfl_xor(whole, off);
    whole = __builtin_amdgcn_readfirstlane(whole);
    // first tile of XCD x: the first one whose predecessors have at least x eighths of the work
    auto first_of = [&](int x) {
      const int64_t target = ((int64_t)whole * per_expert * x + kXcds - 1) / kXcds;
      int64_t before = 0;
      for (int base = 0; base < p.E; base += 64) {
        const int mine = cost_of(base + lane);
        int v = mine;
        for (int off = 1; off < 64; off <<= 1) {
          const int o = __shfl_up(v, off);
          if (lane >= off) v += o;
        }
        const int64_t end = before + (int64_t)v * per_expert;
        const uint64_t past = __ballot(end > target);
        if (past) {
          const int l = __ffsll((unsigned long long)past) - 1;
          const int64_t start = before + (int64_t)(__shfl(v, l) - __shfl(mine, l)) * per_expert;
          const int cost = __shfl(mine, l);
          return (base + l) * per_expert + (int)((target - start + cost - 1) / cost);
        }
        before += (int64_t)__shfl(v, 63) * per_expert;
      }
      return p.E * per_expert;
    };
    from_tile = __builtin_amdgcn_readfirstlane(first_of(xcd));
    last_tile = __builtin_amdgcn_readfirstlane(first_of(xcd + 1));
  } else {
    if (wave == 0) {
      int carry = 0;
      for (int base = 0; base < p.E; base += 64) {
        int row0 = 0, v = 0;
        if (base + lane < p.E) expert_rows(p, base + lane, row0, v);
        v = (v + kTileM - 1) / kTileM;
        for (int off = 1; off < 64; off <<= 1) {
          const int o = __shfl_up(v, off);
          if (lane >= off) v += o;
        }
        if (base + lane < p.E) s_first[base + lane + 1] = carry + v;
        carry += __shfl(v, 63);
      }
      if (lane == 0) s_first[0] = 0;
    }
    __syncthreads();
    m_tiles = __builtin_amdgcn_readfirstlane(s_first[p.E]);
    const int total = m_tiles * NT, chunk = (total + kXcds - 1) / kXcds;
    from_tile = xcd * chunk;
    last_tile = min(total, from_tile + chunk);
  }
  const int first_tile = from_tile + blockIdx.x / kXcds;
  if (first_tile >= last_tile) return;

  // expert, rows, first row and column of a tile: panels of eight m tiles, m fastest
  auto tile_at = [&](int tile) {
    int e = 0, idx, mts;
    if constexpr (kKind == kWeightBack) {
      e = __builtin_amdgcn_readfirstlane(tile / (m_tiles * NT));
      idx = tile - e * m_tiles * NT;
      mts = m_tiles;
    } else {
      const int mtile = __builtin_amdgcn_readfirstlane(tile / NT);
      // the last expert whose first tile is not behind: the experts with a first tile up to it, less one
      for (int base = 1; base <= p.E; base += 64)
        e += __popcll(__ballot(base + lane <= p.E && s_first[min(base + lane, p.E)] <= mtile));
      const int from = __builtin_amdgcn_readfirstlane(s_first[e]);
      idx = tile - from * NT;
      mts = __builtin_amdgcn_readfirstlane(s_first[e + 1]) - from;
    }
    Tile t;
    int count;
    t.e = __builtin_amdgcn_readfirstlane(e);
    expert_rows(p, t.e, t.row0, count);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    count = __builtin_amdgcn_readfirstlane(count);
    // (divisions come out in vector registers, uniform or not)
    const int panel = __builtin_amdgcn_readfirstlane(idx / (8 * NT)), rest = idx - panel * 8 * NT;
    const int high = min(8, mts - panel * 8);
    const int nt = __builtin_amdgcn_readfirstlane(rest / high);
    t.m0 = (panel * 8 + rest - nt * high) * kTileM;
    t.n0 = nt * kCols;
    t.K = kKind == kWeightBack ? count : p.K;
    t.m_left = (kKind == kWeightBack ? p.M : count) - t.m0;
    return t;
  };
  auto units_of = [](int K) { return K > 0 ? (K + kUnitK - 1) / kUnitK : 1; };

  // ---- the cursor that stages
  StageA sa;
  StageB sb;
  int ahead_tile = first_tile, ahead_units = 0, ahead_slot = 0;
  auto advance = [&] {  // to the next tile
    if (ahead_tile >= last_tile) {
      sa.stop();
      sb.stop();
      ahead_units = 1 << 30;
      return;
    }
    const Tile t = tile_at(ahead_tile);
    ahead_tile += per_xcd;
    const int lane = fresh_lane();
    if (lane == 0) s_tile[wave][ahead_slot] = t;
    ahead_slot = ahead_slot + 1 == kAhead ? 0 : ahead_slot + 1;
    ahead_units = units_of(t.K);
    if constexpr (kKind == kWeightBack) {
      sa.start({p.a + ((int64_t)t.row0 * p.lda + t.m0) * 2, p.lda, t.m_left}, t.K, wave, lane);
      sb.start({p.b + ((int64_t)t.row0 * p.ldb + t.n0) * 2, p.ldb, p.N - t.n0}, t.K, wave, lane);
    } else {
      sa.start({p.a + ((int64_t)t.row0 + t.m0) * p.lda * 2, p.lda, t.m_left}, t.K, wave, lane);
      const char* b = p.b + t.e * p.b_expert;
      if constexpr (kDual) {
        const OperandTile up{b + ((int64_t)p.N + t.n0) * p.ldb * 2, p.ldb, p.N - t.n0};
        sb.start({b + (int64_t)t.n0 * p.ldb * 2, p.ldb, p.N - t.n0}, t.K, wave, lane, &up);
      } else if constexpr (kBMContig) {
        sb.start({b + (int64_t)t.n0 * 2, p.ldb, p.N - t.n0}, t.K, wave, lane);
      } else {
        sb.start({b + (int64_t)t.n0 * p.ldb * 2, p.ldb, p.N - t.n0}, t.K, wave, lane);
      }
    }
  };
  const uint32_t lds = (uint32_t)(uintptr_t)s_stage;
  int stage = 0;  // of the unit that is multiplied: the unit kUnits further goes there
  auto issue = [&](int j, int at) {  // the j-th of a unit's DMA instructions
    if (j < StageA::kIssues)
      sa.issue(j, lds + at * kStage, wave);
    else
      sb.issue(j - StageA::kIssues, lds + at * kStage + StageA::kBytes, wave);
    if (j + 1 == kIssues) --ahead_units;
  };

  const int wave_cols = kHalf * 16 * wn;  // this wavefront's first column within the tile
  Reader<kTileM, kAMContig, kWM> ra;
  Reader<kTileN, kBMContig, 1> rb;
  ra.start(wm, lane);
  rb.start(kHalf * wn, lane);

  for (int i = 0; i < kUnits; ++i) {
    if (ahead_units == 0) advance();
#pragma unroll
    for (int j = 0; j < kIssues; ++j) issue(j, i);
  }
  stage_barrier<(kUnits - 1) * kIssues>();

  int slot = 0;
  for (int tile = first_tile; tile < last_tile; tile += per_xcd) {
    Tile t = s_tile[wave][slot];
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    t.m_left = __builtin_amdgcn_readfirstlane(t.m_left);
    t.K = __builtin_amdgcn_readfirstlane(t.K);
    slot = slot + 1 == kAhead ? 0 : slot + 1;

    f32x4_t acc[kMI][kNI];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
      for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // blocks of 16 rows that this wavefront has at all
    const int blocks = (min((t.m_left + 15) / 16, kWM * kMI) - wm + kWM - 1) / kWM;
    auto run = [&](auto count_c) {
      constexpr int kCount = decltype(count_c)::value;
      u32x4_t fa[2][kCount], fb[2][kNI];
      constexpr int kReads = kNI + kCount;
      auto read = [&](int half, int at, int i) {  // the i-th of half a unit's operands
        const uint32_t st = lds + at * kStage;
        if (i < kNI)
          fb[half][i] = rb.get(st + StageA::kBytes, i < kHalf ? i : i - kHalf + kTileN / 32, half);
        else
          fa[half][i - kNI] = ra.get(st, i - kNI, half);
      };
      // Half a unit: groups of products of one row block, in their gaps the reads of the next
      // half's operands.  In the second half also the barrier (the next unit has landed, and every
      // wavefront has read this one) and the DMA into this unit's stage.  The barrier stands behind
      // the first groups: the matrix cores have work while the wavefronts meet.  The order is
      // pinned: left to itself the compiler moves the products behind the barrier and the reads in
      // front of the products.
      auto step = [&](auto half_c, bool behind) {
        constexpr int half = decltype(half_c)::value;
        constexpr int kFirst = half && kCount > 2 ? kCount / 4 : 0;  // groups in front of the barrier, less one
        constexpr int kGaps = kCount - kFirst, kReadGaps = kGaps > 2 ? kGaps - 1 : 1;
        const int here = stage;
        if (half) stage = stage + 1 == kUnits ? 0 : stage + 1;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
#pragma unroll
          for (int j = 0; j < kNI; ++j) acc[i][j] = mfma16<S>(fb[half][j], fa[half][i], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (i < kFirst) continue;
          const int gap = i - kFirst;
          if (half && gap == 0) {
            if (ahead_units == 0) advance();
            if (behind)
              stage_barrier<kPending + kStores>();
            else
              stage_barrier<kPending>();
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int r = gap * kReads / kReadGaps; r < (gap + 1) * kReads / kReadGaps && r < kReads; ++r)
            read(1 - half, stage, r);
          if (half) {
#pragma unroll
            for (int j = gap * kIssues / kGaps; j < (gap + 1) * kIssues / kGaps; ++j) issue(j, here);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
#pragma unroll
      for (int r = 0; r < kReads; ++r) read(0, stage, r);
      // (The last unit of a tile reads the next tile's first, which that tile reads again.  The
      // unit that a tile's first one waits for was staged before the last tile's stores.)
      bool behind = tile != first_tile;
      for (int unit = units_of(t.K); unit > 0; --unit) {
        step(std::integral_constant<int, 0>{}, behind);
        step(std::integral_constant<int, 1>{}, behind);
        behind = false;
      }
    };
    if (blocks > kMI / 2)
      run(std::integral_constant<int, kMI>{});
    else if (kMI < 4 || blocks > kMI / 4)
      run(std::integral_constant<int, kMI / 2>{});
    else
      run(std::integral_constant<int, (kMI < 4 ? 1 : kMI / 4)>{});

    // ---- epilogue: eight consecutive columns of a row per lane and pair of blocks; all lanes
    // execute all loads and stores, those outside at kOutside
    DropKey key{};
    const bool drops = (kKind == kGateUp || kKind == kGateBack) && p.drop.threshold;
    if (drops) key = drop_key(p.drop);
    const int64_t row0 = kKind == kWeightBack ? (int64_t)t.e * p.M + t.m0 : (int64_t)t.row0 + t.m0;
    const __amdgpu_buffer_rsrc_t out = open_resource(p.out + (row0 * p.ldo + t.n0) * 2);
    const int here = fresh_lane();
    const int col0 = wave_cols + eight_column(here);  // within the tile
    auto row_of = [&](int i) { return 16 * (kWM * i + wm) + (here & 15); };
    auto offset_of = [&](int row, int col, int ld) {
      return row < t.m_left && t.n0 + col < p.N ? ((uint32_t)row * (uint32_t)ld + (uint32_t)col) * 2u : kOutside;
    };
    if constexpr (kKind == kGateUp) {
      const __amdgpu_buffer_rsrc_t gate = open_resource(p.gu + (row0 * p.ldgu + t.n0) * 2);
      const __amdgpu_buffer_rsrc_t up = open_resource(p.gu + (row0 * p.ldgu + p.N + t.n0) * 2);
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        const int row = row_of(i);
        float g[8], u[8];
        eight_columns(acc[i][0], acc[i][1], g);
        eight_columns(acc[i][2], acc[i][3], u);
        if (p.gu) {
          const uint32_t at = offset_of(row, col0, p.ldgu);
          store16(pack8<S>(g), gate, at);
          store16(pack8<S>(u), up, at);
        }
        u32x4_t n{};
        if (drops) n = drop_numbers(key, p.drop.site, (uint32_t)(row0 + row), (uint32_t)(t.n0 + col0) >> 3);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float slope;
          g[c] = activate(p.activation, g[c], slope) * u[c];
          if (drops) g[c] = drop_keeps(n, c, p.drop.threshold) ? g[c] * p.drop.scale : 0.f;
        }
        store16(pack8<S>(g), out, offset_of(row, col0, p.ldo));
      }
    } else if constexpr (kKind == kGateBack) {
      // g and u of two row blocks are requested at once, before the first is used
      constexpr int kAtOnce = 2;
      const __amdgpu_buffer_rsrc_t gate = open_resource(p.gu + (row0 * p.ldgu + t.n0) * 2);
      const __amdgpu_buffer_rsrc_t up = open_resource(p.gu + (row0 * p.ldgu + p.N + t.n0) * 2);
      const __amdgpu_buffer_rsrc_t out_up = open_resource(p.out + (row0 * p.ldo + p.N + t.n0) * 2);
#pragma unroll
      for (int i0 = 0; i0 < kMI; i0 += kAtOnce) {
        Raw<S> rg[kAtOnce][2], ru[kAtOnce][2];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t at = offset_of(row_of(i0 + i), col0 + 32 * j, p.ldgu);
            rg[i][j].w[0] = load16(gate, at);
            ru[i][j].w[0] = load16(up, at);
          }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int row = row_of(i0 + i), col = col0 + 32 * j;
            float v[8], g[8], u[8];
            eight_columns(acc[i0 + i][2 * j], acc[i0 + i][2 * j + 1], v);
            unpack(rg[i][j], g);
            unpack(ru[i][j], u);
            u32x4_t n{};
            if (drops) n = drop_numbers(key, p.drop.site, (uint32_t)(row0 + row), (uint32_t)(t.n0 + col) >> 3);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              // (what is dropped is selected away: its g and u may be infinite)
              const bool keep = !drops || drop_keeps(n, c, p.drop.threshold);
              if (drops) v[c] *= p.drop.scale;
              float slope;
              const float act = activate(p.activation, g[c], slope);
              g[c] = keep ? v[c] * u[c] * slope : 0.f;
              u[c] = keep ? v[c] * act : 0.f;
            }
            const uint32_t to = offset_of(row, col, p.ldo);
            store16(pack8<S>(g), out, to);
            store16(pack8<S>(u), out_up, to);
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v[8];
          eight_columns(acc[i][2 * j], acc[i][2 * j + 1], v);
          store16(pack8<S>(v), out, offset_of(row_of(i), col0 + 32 * j, p.ldo));
        }
    }
  }
  stage_barrier<0>();  // no DMA outlives the workgroup's LDS
}

// Few rows per expert: gate/up or down by workgroups of 16 columns (16 gate and 16 up columns), whose
// eight wavefronts share K and add their sums in LDS in wavefront order.  Weights go from memory to
// the matrix cores' registers, nothing is staged.  A pass takes four 64-k pieces of each wavefront;
// the compiler puts their products between their loads, so that three loads are in flight at its
// start (gated; four otherwise) and nine at most, in 90 registers.  Bound by that latency at one
// expert (a row of d = 2048, I = 1024: 7.1 and 4.5 us, 10.8 for the call; 20 and 11 by tiles of 64
// rows, which stage 32 units one behind the other), by memory at large ones (d = 4096, I = 14336: 50
// and 24 us, 4.7 TB/s).  An expert's weights are read again for every 16 of its rows.
template <typename S, bool kDual>
__global__ __launch_bounds__(512) void k_few(ProductDev p) {
  constexpr int kBlocks = kDual ? 2 : 1, kAtOnce = 4, kWaves = 8;
  __shared__ float s_part[kWaves][kBlocks][16][17];
  const int lane = lane_id(), i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int row0, count;
  const int e = blockIdx.y, n0 = blockIdx.x * 16;
  expert_rows(p, e, row0, count);
  const char* w[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)  // columns past the last one read that one
    w[b] = p.b + e * p.b_expert + ((int64_t)b * p.N + min(n0 + i, p.N - 1)) * p.ldb * 2;
  DropKey key{};
  const bool drops = kDual && p.drop.threshold;
  if (drops) key = drop_key(p.drop);
  for (int m0 = 0; m0 < count; m0 += 16) {
    const char* x = p.a + ((int64_t)row0 + min(m0 + i, count - 1)) * p.lda * 2;
    f32x4_t acc[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave * kUnitK; k0 < p.K; k0 += kAtOnce * kWaves * kUnitK) {
      u32x4_t fx[kAtOnce][2], fw[kAtOnce][2][kBlocks];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + u * kWaves * kUnitK + 32 * h + 8 * q;
          const int64_t at = 2 * (int64_t)min(k, p.K - 8);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) fw[u][h][b] = *reinterpret_cast<const u32x4_t*>(w[b] + at);
          fx[u][h] = *reinterpret_cast<const u32x4_t*>(x + at);
        }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t inside = k0 + u * kWaves * kUnitK + 32 * h + 8 * q < p.K ? 0xFFFFFFFFu : 0u;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            acc[b] = mfma16<S>(fw[u][h][b] & inside, fx[u][h] & inside, acc[b]);
        }
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) s_part[wave][b][i][4 * q + r] = acc[b][r];
    __syncthreads();
    const int m = threadIdx.x >> 4, n = threadIdx.x & 15, col = n0 + n;
    if (threadIdx.x < 256 && m0 + m < count && col < p.N) {
      float v[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        v[b] = 0.f;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) v[b] += s_part[o][b][m][n];
      }
      const int64_t row = (int64_t)row0 + m0 + m;
      if constexpr (kDual) {
        if (p.gu) {
          S* at = reinterpret_cast<S*>(p.gu) + row * p.ldgu + col;
          store_one(at, v[0]);
          store_one(at + p.N, v[1]);
        }
        float slope;
        v[0] = activate(p.activation, v[0], slope) * v[1];
        if (drops) {
          const u32x4_t numbers = drop_numbers(key, p.drop.site, (uint32_t)row, (uint32_t)col >> 3);
          const uint32_t word = (col & 4) ? ((col & 2) ? numbers[3] : numbers[2]) : ((col & 2) ? numbers[1] : numbers[0]);
          v[0] = ((col & 1) ? word >> 16 : word & 0xFFFFu) >= p.drop.threshold ? v[0] * p.drop.scale : 0.f;
        }
      }
      store_one(reinterpret_cast<S*>(p.out) + row * p.ldo + col, v[0]);
    }
    __syncthreads();
  }
}

// The time of a product by tiles of a shape, in microseconds: tiles in rounds, a round of so much
// per unit of k and so much for its start and end.  Measured, by 256 x 256, 128 x 256, 128 x 128 and
// 64 x 256, the chosen one in brackets:
//   E = 13, R = 2331, d = 1000, I = 712    gate/up  41 (31) 34 37     dx  39 27 23 (20)
//   E = 1, R = 4096, d = 2048, I = 8192    gate/up  (250) 296 338 417   dx  374 (259) 285 343
//   E = 64, R = 32768, d = 2048, I = 1024  gate/up  (340) 305 365 420   down  (186) 171 204 230
//   E = 8, R = 2048, d = 4096, I = 14336   gate/up  (588) 558 680 760   down  (390) 420 485 505
//   E = 1, R = 32768, d = 1024, I = 512    dW13  601 (372) 428          dWd  673 (420) 433
// Where rows, columns or experts leave CUs idle the smaller tiles win.  The experts' unequal rows are
// not in the model: there 128 x 256 wins where 256 x 256 is chosen, by an eighth at most above, by a
// fifth at E = 8, R = 32768, d = 1024, I = 512 (dh 99 us by 256 x 256, 88 by 128 x 256, 82 by 128 x 128).
template <typename Sh>
static double product_us(const ProductDev& p, bool weights, bool gated) {
  const double per_unit = Sh::kTileM == 256 ? 1.5 : Sh::kTileM == 64 ? 0.7 : Sh::kTileN == 256 ? 1.05 : 1.15;
  const double ends = Sh::kTileM == 256 ? 14 : Sh::kTileM == 64 ? 5 : 7;
  const double used = std::min(p.E, p.R), rows = (double)p.R / Sh::kTileM;
  const double m_tiles = weights    ? (double)p.E * ceil_div(p.M, Sh::kTileM)
                         : p.E == 1 ? std::ceil(rows)
                                    : std::max(rows + 0.5 * used, 0.9 * used);
  const double k = weights ? (double)p.R / p.E : p.K;
  const double rounds = m_tiles * ceil_div(p.N, gated ? Sh::kTileN / 2 : Sh::kTileN) / (256 * Sh::kPerCu);
  return (rounds <= 1 ? 1 : rounds + 0.5) * (std::ceil(k / kUnitK) * per_unit + ends);
}

template <int kKind>
static void launch_product(const ProductDev& p, int dtype, hipStream_t s) {
  constexpr bool weights = kKind == kWeightBack, gated = kKind == kGateUp;
  auto launch = [&](auto type, auto shape) {
    using S = decltype(type);
    using Sh = decltype(shape);
    const int64_t cols = gated ? Sh::kTileN / 2 : Sh::kTileN, tm = Sh::kTileM;
    const int64_t m_tiles = weights ? p.E * ceil_div(p.M, tm) : p.R / tm + std::min(p.E, p.R);
    const int64_t tiles = m_tiles * ceil_div(p.N, cols);
    const unsigned grid = (unsigned)std::min<int64_t>(256 * Sh::kPerCu, ceil_div(tiles, kXcds) * kXcds);
    hipLaunchKernelGGL((k_product<S, kKind, Sh>), dim3(grid), dim3(64 * Sh::kWaves), 0, s, p);
  };
  const double t256 = product_us<Shape256>(p, weights, gated), t128 = product_us<Shape128>(p, weights, gated);
  const double half = product_us<ShapeHalf>(p, weights, gated);
  const double t64 = weights ? 1e30 : product_us<Shape64>(p, weights, gated);
  const double best = std::min(std::min(t256, t128), std::min(half, t64));
  auto go = [&](auto type) {
    using S = decltype(type);
    if constexpr (kKind == kGateUp || kKind == kDown) {
      // At most 16 rows per expert on average: where tiles of 64 rows leave CUs idle, or where a
      // workgroup has 256 KB of weights to read.  Measured, gate/up and down in us, this kernel
      // against tiles of 64 rows: one row of d = 2048, I = 1024 7 and 5 against 20 and 11; E = 8,
      // R = 16, d = 4096, I = 14336 310 and 151 against 316 and 192; E = 8, d = 2048, I = 1024, 2, 8 and
      // 16 rows per expert on average 19 and 13, 22 and 15, 30 and 22 against 27, 28, 28 and 15; E = 64,
      // 2 rows each (tiles are taken) 96 and 66 against 102 and 40.  What the rule does not see: rows
      // on one expert, read 16 at a time (all 128 rows on one of the eight 50 and 33 against 22 and
      // 13), and many experts with a long K, where tiles win (E = 64, d = 4096, gate/up, 2 and 16 rows
      // per expert 163 and 304 against 150 and 223, all 1024 rows on one 710 against 40).
      const int64_t tiles = std::min(p.E, p.R) * ceil_div(p.N, gated ? Shape64::kTileN / 2 : Shape64::kTileN);
      if (p.R <= 16 * (int64_t)p.E && (tiles <= 256 || (gated ? 32 : 16) * (int64_t)p.K >= 1 << 17)) {
        hipLaunchKernelGGL((k_few<S, gated>), dim3((unsigned)ceil_div(p.N, 16), p.E), dim3(512), 0, s, p);
        return;
      }
    }
    if (t256 == best)
      launch(type, Shape256{});
    else if (t128 == best)
      launch(type, Shape128{});
    else if (half == best)
      launch(type, ShapeHalf{});
    else if constexpr (!weights)
      launch(type, Shape64{});
  };
  if (dtype == MOE_BF16)
    go(bf16_row_t{});
  else
    go(_Float16{});
}

constexpr int kFfnMaxSize = 1 << 16;    // d and I
constexpr int kFfnMaxStride = 1 << 20;  // elements between rows: a tile's rows lie within 2^31 bytes

static int check_ffn(const char* fn, const moe_gated_ffn_args* a) {
  MOE_CHECK_ARG(a != nullptr, MOE_ERR_INVALID_ARG, "%s: args is NULL", fn);
  MOE_CHECK_ARG(a->dtype == MOE_BF16 || a->dtype == MOE_FP16, MOE_ERR_INVALID_ARG, "%s: bad dtype %d (bf16 or fp16)", fn,
                a->dtype);
  MOE_CHECK_ARG(a->activation == MOE_ACT_SILU || a->activation == MOE_ACT_GELU, MOE_ERR_INVALID_ARG,
                "%s: bad activation %d", fn, a->activation);
  MOE_CHECK_ARG(a->num_rows >= 0 && a->d > 0 && a->I > 0 && a->E > 0, MOE_ERR_INVALID_ARG,
                "%s: bad sizes num_rows=%d d=%d I=%d E=%d", fn, a->num_rows, a->d, a->I, a->E);
  MOE_CHECK_ARG(a->d % 8 == 0 && a->I % 8 == 0 && a->d <= kFfnMaxSize && a->I <= kFfnMaxSize &&
                    a->E <= MOE_MAX_EXPERTS && a->num_rows <= (1 << 24),
                MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: unsupported num_rows=%d d=%d I=%d E=%d (d and I multiples of 8 up to %d, E <= %d, num_rows <= 2^24)",
                fn, a->num_rows, a->d, a->I, a->E, kFfnMaxSize, MOE_MAX_EXPERTS);
  MOE_CHECK_ARG(a->expert_offsets ? ((uintptr_t)a->expert_offsets % 4) == 0 : a->E == 1, MOE_ERR_INVALID_ARG,
                "%s: expert_offsets is misaligned, or NULL for E=%d", fn, a->E);
  return check_dropout(fn, a->drop_p, a->drop_state, a->drop_site);
}

static int check_matrix(const char* fn, const char* name, const void* p, int64_t stride, int64_t least, bool wanted) {
  if (!wanted) return MOE_OK;
  MOE_CHECK_ARG(p && ((uintptr_t)p % 16) == 0, MOE_ERR_INVALID_ARG, "%s: %s is NULL or not 16-byte aligned", fn, name);
  MOE_CHECK_ARG(stride >= least && stride % 8 == 0, MOE_ERR_INVALID_ARG,
                "%s: stride %lld of %s below %lld or no multiple of 8", fn, (long long)stride, name, (long long)least);
  MOE_CHECK_ARG(stride <= kFfnMaxStride, MOE_ERR_UNSUPPORTED_SHAPE, "%s: stride %lld of %s above 2^20", fn,
                (long long)stride, name);
  return MOE_OK;
}

static ProductDev product(const moe_gated_ffn_args* a) {
  ProductDev p{};
  p.R = a->num_rows;
  p.E = a->E;
  p.offsets = a->expert_offsets;
  p.activation = a->activation;
  p.drop = drop_dev(a->drop_p, a->drop_state, a->drop_site);
  return p;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_gated_ffn(const moe_gated_ffn_args* a, void* gu, int64_t gu_stride, void* h, int64_t h_stride, void* y,
                             int64_t y_stride, void* stream) {
  clear_error();
  const char* fn = "moe_gated_ffn";
  int rc = check_ffn(fn, a);
  if (rc || a->num_rows == 0) return rc;
  const int64_t d = a->d, I = a->I;
  if ((rc = check_matrix(fn, "rows", a->rows, a->rows_stride, d, true))) return rc;
  if ((rc = check_matrix(fn, "w13", a->w13, d, d, true))) return rc;
  if ((rc = check_matrix(fn, "w2", a->w2, I, I, y != nullptr))) return rc;
  if ((rc = check_matrix(fn, "gu", gu, gu_stride, 2 * I, gu != nullptr))) return rc;
  if ((rc = check_matrix(fn, "h", h, h_stride, I, true))) return rc;
  if ((rc = check_matrix(fn, "y", y, y_stride, d, y != nullptr))) return rc;
  hipStream_t s = (hipStream_t)stream;
  timing_begin(K_GATED_FFN, s);
  ProductDev p = product(a);
  p.a = static_cast<const char*>(a->rows);
  p.lda = (int)a->rows_stride;
  p.b = static_cast<const char*>(a->w13);
  p.ldb = a->d;
  p.b_expert = 2 * I * d * 2;
  p.N = a->I;
  p.K = a->d;
  p.out = static_cast<char*>(h);
  p.ldo = (int)h_stride;
  p.gu = static_cast<char*>(gu);
  p.ldgu = (int)gu_stride;
  launch_product<kGateUp>(p, a->dtype, s);
  if (y) {
    ProductDev q = product(a);
    q.a = static_cast<const char*>(h);
    q.lda = (int)h_stride;
    q.b = static_cast<const char*>(a->w2);
    q.ldb = a->I;
    q.b_expert = d * I * 2;
    q.N = a->d;
    q.K = a->I;
    q.out = static_cast<char*>(y);
    q.ldo = (int)y_stride;
    launch_product<kDown>(q, a->dtype, s);
  }
  timing_end(K_GATED_FFN, s);
  return check_launch(fn);
}

extern "C" int64_t moe_gated_ffn_backward_workspace_bytes(int num_rows, int d, int I, int E) {
  if (num_rows < 0 || d <= 0 || I <= 0 || E <= 0) return -1;
  if (d % 8 || I % 8 || d > kFfnMaxSize || I > kFfnMaxSize || E > MOE_MAX_EXPERTS || num_rows > (1 << 24)) return -1;
  return ceil_div((int64_t)num_rows * 2 * I * 2, 256) * 256;
}

extern "C" int moe_gated_ffn_backward(const moe_gated_ffn_args* a, const moe_gated_ffn_grads* g, void* stream) {
  clear_error();
  const char* fn = "moe_gated_ffn_backward";
  int rc = check_ffn(fn, a);
  if (rc) return rc;
  MOE_CHECK_ARG(g != nullptr, MOE_ERR_INVALID_ARG, "%s: grads is NULL", fn);
  MOE_CHECK_ARG(g->drows || g->dw13 || g->dw2 || a->num_rows == 0, MOE_ERR_INVALID_ARG, "%s: no gradient is wanted", fn);
  const int64_t d = a->d, I = a->I;
  const bool some = a->num_rows > 0, through = g->drows || g->dw13;
  if ((rc = check_matrix(fn, "dy", g->dy, g->dy_stride, d, some))) return rc;
  if ((rc = check_matrix(fn, "rows", a->rows, a->rows_stride, d, some && g->dw13))) return rc;
  if ((rc = check_matrix(fn, "w13", a->w13, d, d, some && g->drows))) return rc;
  if ((rc = check_matrix(fn, "w2", a->w2, I, I, some && through))) return rc;
  if ((rc = check_matrix(fn, "gu", g->gu, g->gu_stride, 2 * I, some && through))) return rc;
  if ((rc = check_matrix(fn, "h", g->h, g->h_stride, I, some && g->dw2))) return rc;
  if ((rc = check_matrix(fn, "drows", g->drows, g->drows_stride, d, some && g->drows))) return rc;
  if ((rc = check_matrix(fn, "dw13", g->dw13, d, d, g->dw13 != nullptr))) return rc;
  if ((rc = check_matrix(fn, "dw2", g->dw2, I, I, g->dw2 != nullptr))) return rc;
  const int64_t need = moe_gated_ffn_backward_workspace_bytes(a->num_rows, a->d, a->I, a->E);
  MOE_CHECK_ARG(!some || !through ||
                    (g->workspace && g->workspace_bytes >= need && ((uintptr_t)g->workspace % 256) == 0),
                MOE_ERR_WORKSPACE, "%s: workspace of %lld bytes < %lld needed, NULL or misaligned", fn,
                (long long)g->workspace_bytes, (long long)need);
  if (!some && !g->dw13 && !g->dw2) return MOE_OK;
  hipStream_t s = (hipStream_t)stream;
  timing_begin(K_GATED_FFN_BWD, s);
  char* dgu = static_cast<char*>(g->workspace);
  if (some && through) {
    ProductDev p = product(a);
    p.a = static_cast<const char*>(g->dy);
    p.lda = (int)g->dy_stride;
    p.b = static_cast<const char*>(a->w2);
    p.ldb = a->I;
    p.b_expert = d * I * 2;
    p.N = a->I;
    p.K = a->d;
    p.out = dgu;
    p.ldo = 2 * a->I;
    p.gu = static_cast<char*>(const_cast<void*>(g->gu));
    p.ldgu = (int)g->gu_stride;
    launch_product<kGateBack>(p, a->dtype, s);
  }
  if (some && g->drows) {
    ProductDev p = product(a);
    p.a = dgu;
    p.lda = 2 * a->I;
    p.b = static_cast<const char*>(a->w13);
    p.ldb = a->d;
    p.b_expert = 2 * I * d * 2;
    p.N = a->d;
    p.K = 2 * a->I;
    p.out = static_cast<char*>(g->drows);
    p.ldo = (int)g->drows_stride;
    launch_product<kRowsBack>(p, a->dtype, s);
  }
  if (g->dw13) {
    ProductDev p = product(a);
    p.a = dgu;
    p.lda = 2 * a->I;
    p.b = static_cast<const char*>(a->rows);
    p.ldb = (int)a->rows_stride;
    p.M = 2 * a->I;
    p.N = a->d;
    p.out = static_cast<char*>(g->dw13);
    p.ldo = a->d;
    launch_product<kWeightBack>(p, a->dtype, s);
  }
  if (g->dw2) {
    ProductDev p = product(a);
    p.a = static_cast<const char*>(g->dy);
    p.lda = (int)g->dy_stride;
    p.b = static_cast<const char*>(g->h);
    p.ldb = (int)g->h_stride;
    p.M = a->d;
    p.N = a->I;
    p.out = static_cast<char*>(g->dw2);
    p.ldo = a->I;
    launch_product<kWeightBack>(p, a->dtype, s);
  }
  timing_end(K_GATED_FFN_BWD, s);
  return check_launch(fn);
}

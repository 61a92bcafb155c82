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
#include "rows.hpp"

namespace moe {

constexpr int kRbTokens = 16;      // tokens per workgroup of the logits' gradient
constexpr int kRbCols = 128;       // columns of d per wavefront
constexpr int kRbTokenBlocks = 2;  // token blocks of 16 per wavefront of dx

struct RouteBackDev {
  const uint16_t *x, *w;
  int T, d, E, k, renormalize;
  int64_t Tp;  // T rounded up to 32
  int Ep;      // E rounded up to 32 (E <= 32) or 64
  const float* logits;
  const int32_t* ids;
  const float *weights, *dweights, *dlogits;
  const uint16_t* dx_add;
  uint16_t* dx;
  float* dw;
  uint16_t* g_rows;  // [2][Tp][Ep]: G in two bf16 parts
  uint16_t* g_cols;  // [3][Ep][Tp]: G^T in three
  float* part;       // [splits][E][d] or null
  int splits;
};

// floats per token in LDS: odd, so that a column's tokens lie in different banks, but
// at most 64 KiB for all tokens
__host__ __device__ inline int rb_row_floats(int Ep) { return Ep < 1024 ? Ep + 1 : Ep; }
static_assert(kRbTokens * 1024 * 4 <= 65536 && MOE_MAX_EXPERTS <= 1024, "LDS of k_route_dlogits");

// The gradient of the logits of kRbTokens tokens, split and stored both ways: a wavefront
// per token, its E <= 64 kEL logits (read once) in the lanes' registers.
template <int kEL>
__global__ __launch_bounds__(64 * kRbTokens) void k_route_dlogits(RouteBackDev a) {
  extern __shared__ float g[];  // [kRbTokens][ld]
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kRbTokens, t = t0 + wave;
  const int ld = rb_row_floats(a.Ep);
  float* row = g + wave * ld;
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
    // the selected experts' own values, through LDS to the lanes that hold them
#pragma unroll
    for (int i = 0; i < kEL; ++i)
      if (lane + 64 * i < a.Ep) row[lane + 64 * i] = v[i];
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) row[id] = w * (dw - s);
    __builtin_amdgcn_wave_barrier();
    if (a.dlogits)
#pragma unroll
      for (int i = 0; i < kEL; ++i)
        if (lane + 64 * i < a.E) row[lane + 64 * i] += add[i];
  } else {
    for (int e = lane; e < a.Ep; e += 64) row[e] = 0.f;
  }
  __syncthreads();
  // rows: two parts
  const int64_t plane = a.Tp * a.Ep;
  for (int i = threadIdx.x; i < kRbTokens * a.Ep / 2; i += 64 * kRbTokens) {
    const int r = i / (a.Ep / 2), e = i % (a.Ep / 2) * 2;
    const float v0 = g[r * ld + e], v1 = g[r * ld + e + 1];
    const uint32_t hi = pack_bf16x2(v0, v1);
    const uint32_t lo = pack_bf16x2(v0 - __uint_as_float(hi << 16), v1 - __uint_as_float(hi & 0xFFFF0000u));
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.g_rows + (t0 + r) * a.Ep + e);
    dst[0] = hi;
    dst[plane / 2] = lo;
  }
  // columns: three parts, eight tokens at a time
  for (int i = threadIdx.x; i < a.Ep * (kRbTokens / 8); i += 64 * kRbTokens) {
    const int e = i / (kRbTokens / 8), r = i % (kRbTokens / 8) * 8;
    u32x4_t p[3];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v0 = g[(r + 2 * q) * ld + e], v1 = g[(r + 2 * q + 1) * ld + e];
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        p[s][q] = pack_bf16x2(v0, v1);
        v0 -= __uint_as_float(p[s][q] << 16);
        v1 -= __uint_as_float(p[s][q] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) *reinterpret_cast<u32x4_t*>(a.g_cols + s * plane + e * a.Tp + t0 + r) = p[s];
  }
}

// Eight rows, r0 .. r0 + 7 (clamped to the last), of a lane's eight columns ...
struct Block8 {
  u32x4_t row[8];
};
__device__ __forceinline__ Block8 load_block8(const uint16_t* m, int64_t r0, int64_t last, int64_t stride) {
  Block8 b;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t q = r0 + r < last ? r0 + r : last;
    b.row[r] = *reinterpret_cast<const u32x4_t*>(m + q * stride);
  }
  return b;
}
// ... and column c of them, as eight k of an MFMA operand
__device__ __forceinline__ bf16x8_t column(const Block8& b, int c) {
  u32x4_t v;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    v[p] = __builtin_amdgcn_perm(b.row[2 * p + 1][c >> 1], b.row[2 * p][c >> 1], (c & 1) ? 0x07060302u : 0x05040100u);
  return as_bf16x8(v);
}

constexpr int kRbWaves = 8;  // per workgroup of the products
typedef float rb_sums_t[16][kRbCols + 4];

// dW: a workgroup sums 16 EB experts x 128 columns over its share of the tokens, its
// wavefronts each over steps of 32 tokens of their own; they meet in LDS.
template <int EB>
__device__ __forceinline__ void route_dw(const RouteBackDev& a, int block, rb_sums_t* sums) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int n = lane & 15, kq = lane >> 4;
  const int chunks = (a.d + kRbCols - 1) / kRbCols, tiles = (a.E + 16 * EB - 1) / (16 * EB);
  const int c0 = block % chunks * kRbCols;
  const int e0 = block / chunks % tiles * 16 * EB;
  const int split = block / chunks / tiles;
  const int col = c0 + 8 * n < a.d ? c0 + 8 * n : 0;  // columns past the end: summed and not stored
  const int64_t steps = a.Tp / 32, plane = a.Tp * a.Ep;
  const int64_t stride = (int64_t)kRbWaves * a.splits;
  f32x4_t acc[EB][8];
#pragma unroll
  for (int b = 0; b < EB; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int64_t st = split * kRbWaves + wave;
  Block8 next;
  if (st < steps) next = load_block8(a.x + col, st * 32 + 8 * kq, a.T - 1, a.d);
  for (; st < steps; st += stride) {
    const Block8 x = next;
    u32x4_t gf[EB][3];
#pragma unroll
    for (int b = 0; b < EB; ++b)
#pragma unroll
      for (int s = 0; s < 3; ++s)
        gf[b][s] = *reinterpret_cast<const u32x4_t*>(a.g_cols + s * plane + (int64_t)(e0 + 16 * b + n) * a.Tp +
                                                     st * 32 + 8 * kq);
    if (st + stride < steps) next = load_block8(a.x + col, (st + stride) * 32 + 8 * kq, a.T - 1, a.d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x8_t xf = column(x, i);
#pragma unroll
      for (int b = 0; b < EB; ++b)
#pragma unroll
        for (int s = 0; s < 3; ++s) acc[b][i] = mfma16x16x32(as_bf16x8(gf[b][s]), xf, acc[b][i]);
    }
  }
  float* out = a.splits > 1 ? a.part + (int64_t)split * a.E * a.d : a.dw;
#pragma unroll
  for (int b = 0; b < EB; ++b) {
    if (e0 + 16 * b >= a.E) break;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float* p = &sums[wave][4 * kq + q][8 * n];
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{acc[b][0][q], acc[b][1][q], acc[b][2][q], acc[b][3][q]};
      *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{acc[b][4][q], acc[b][5][q], acc[b][6][q], acc[b][7][q]};
    }
    __syncthreads();
    static_assert(kRbWaves * 64 == 16 * kRbCols / 4, "four columns of a row per thread");
    const int r = threadIdx.x / (kRbCols / 4), c = threadIdx.x % (kRbCols / 4) * 4;
    const int e = e0 + 16 * b + r;
    if (e < a.E && c0 + c < a.d) {
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(&sums[0][r][c]);
#pragma unroll
      for (int w = 1; w < kRbWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(&sums[w][r][c]);
      *reinterpret_cast<f32x4_t*>(out + (int64_t)e * a.d + c0 + c) = v;
    }
  }
}

// dx: a wavefront computes 16 kRbTokenBlocks tokens x 128 columns, 32 experts a step.
__device__ __forceinline__ void route_dx(const RouteBackDev& a, int block) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int n = lane & 15, kq = lane >> 4;
  const int chunks = (a.d + kRbCols - 1) / kRbCols;
  const int c0 = block % chunks * kRbCols;
  const int64_t t0 = ((int64_t)(block / chunks) * kRbWaves + wave) * 16 * kRbTokenBlocks;
  if (t0 >= a.T) return;
  const bool stored = c0 + 8 * n < a.d;
  const int col = stored ? c0 + 8 * n : 0;
  const int64_t plane = a.Tp * a.Ep;
  u32x4_t add[kRbTokenBlocks][4];
#pragma unroll
  for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t t = t0 + 16 * b + 4 * kq + q;
      add[b][q] = u32x4_t{0, 0, 0, 0};
      if (a.dx_add) add[b][q] = *reinterpret_cast<const u32x4_t*>(a.dx_add + (t < a.T ? t : a.T - 1) * a.d + col);
    }
  f32x4_t acc[kRbTokenBlocks][8];
#pragma unroll
  for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint16_t* grow[kRbTokenBlocks];
#pragma unroll
  for (int b = 0; b < kRbTokenBlocks; ++b) {
    const int64_t t = t0 + 16 * b + n;
    grow[b] = a.g_rows + (t < a.Tp ? t : a.Tp - 1) * a.Ep + 8 * kq;
  }
  const int last = (a.E + 31) / 32 * 32;
  Block8 next = load_block8(a.w + col, 8 * kq, a.E - 1, a.d);
  u32x4_t gnext[kRbTokenBlocks][2];
  auto request = [&](int e) {
#pragma unroll
    for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
      for (int s = 0; s < 2; ++s) gnext[b][s] = *reinterpret_cast<const u32x4_t*>(grow[b] + e + s * plane);
  };
  request(0);
  for (int e = 0; e < last; e += 32) {
    const Block8 w = next;
    u32x4_t gf[kRbTokenBlocks][2];
#pragma unroll
    for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
      for (int s = 0; s < 2; ++s) gf[b][s] = gnext[b][s];
    if (e + 32 < last) {
      next = load_block8(a.w + col, e + 32 + 8 * kq, a.E - 1, a.d);
      request(e + 32);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x8_t wf = column(w, i);
#pragma unroll
      for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[b][i] = mfma16x16x32(as_bf16x8(gf[b][s]), wf, acc[b][i]);
    }
  }
  if (!stored) return;
#pragma unroll
  for (int b = 0; b < kRbTokenBlocks; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t t = t0 + 16 * b + 4 * kq + q;
      if (t >= a.T) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t p = add[b][q][i >> 1];
        v[i] = acc[b][i][q] + __uint_as_float((i & 1) ? (p & 0xFFFF0000u) : (p << 16));
      }
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<u32x4_t*>(a.dx + t * a.d + c0 + 8 * n) = o;
    }
}

// Both products in one launch: the first dw_blocks workgroups sum dW, the others dx.
template <int EB>
__global__ __launch_bounds__(64 * kRbWaves) void k_route_products(RouteBackDev a, int dw_blocks) {
  __shared__ rb_sums_t sums[kRbWaves];
  if ((int)blockIdx.x < dw_blocks)
    route_dw<EB>(a, blockIdx.x, sums);
  else
    route_dx(a, blockIdx.x - dw_blocks);
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
  int64_t Tp, rows_bytes, cols_bytes, part_bytes, total;
  int Ep, EB, splits;
};

static RouteBackPlan route_back_plan(int T, int d, int E) {
  RouteBackPlan p;
  p.Tp = ceil_div(T, 32) * 32;
  p.Ep = E <= 32 ? 32 : (int)ceil_div(E, 64) * 64;
  p.EB = E <= 16 ? 1 : E <= 32 ? 2 : 4;
  const int64_t tiles = ceil_div(d, kRbCols) * ceil_div(E, 16 * p.EB);
  const int64_t most = std::max<int64_t>(1, ceil_div(p.Tp / 32, kRbWaves));
  p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, ceil_div(256, tiles)));
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  p.rows_bytes = up(2 * p.Tp * p.Ep * 2);
  p.cols_bytes = up(3 * p.Tp * p.Ep * 2);
  p.part_bytes = p.splits > 1 ? up((int64_t)p.splits * E * d * 4) : 0;
  p.total = p.rows_bytes + p.cols_bytes + p.part_bytes;
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
  v.g_rows = reinterpret_cast<uint16_t*>(ws);
  v.g_cols = reinterpret_cast<uint16_t*>(ws + p.rows_bytes);
  v.part = reinterpret_cast<float*>(ws + p.rows_bytes + p.cols_bytes);
  v.splits = p.splits;
  timing_begin(K_ROUTE_BWD, s);
  const int per_lane = (int)ceil_div(p.Ep, 64);
  auto dlogits = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.Tp / kRbTokens)), dim3(64 * kRbTokens),
                       kRbTokens * rb_row_floats(p.Ep) * sizeof(float), s, v);
  };
  if (per_lane <= 1)
    dlogits(k_route_dlogits<1>);
  else if (per_lane <= 4)
    dlogits(k_route_dlogits<4>);
  else
    dlogits(k_route_dlogits<16>);
  const int64_t chunks = ceil_div(a->d, kRbCols);
  const int64_t dw_blocks = a->dw_router ? chunks * ceil_div(a->E, 16 * p.EB) * p.splits : 0;
  const int64_t dx_blocks = a->dx ? chunks * ceil_div(a->T, 16 * kRbTokenBlocks * kRbWaves) : 0;
  auto products = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(dw_blocks + dx_blocks)), dim3(64 * kRbWaves), 0, s, v, (int)dw_blocks);
  };
  if (p.EB == 1)
    products(k_route_products<1>);
  else if (p.EB == 2)
    products(k_route_products<2>);
  else
    products(k_route_products<4>);
  if (a->dw_router && p.splits > 1) {
    const int64_t count = (int64_t)a->E * a->d;
    hipLaunchKernelGGL(k_route_dw_sum, dim3((unsigned)ceil_div(count, 1024)), dim3(256), 0, s, v.part, p.splits, count,
                       a->dw_router);
  }
  timing_end(K_ROUTE_BWD, s);
  return check_launch("moe_route_backward");
}

// moe_block_norm: the norm behind a block with its gate, the scaled residual and the
// norm before the next block, and its gradient (ExactMoE, page "Every Expert Counts:
// ExactMoE for Memory-Efficient W4A16 Inference", Abstract: the normalization layers
// around the routed experts stay in BF16).
//
// One row, with r_y = 1 / sqrt(mean(y^2) + eps) and r_h likewise of h:
//   z = r_y y v_out,  h = a x + g z,  n = r_h h v_in.
// Gradient, with u = dn v_in and the normalised rows yn = r_y y, hn = r_h h:
//   D  = dh + r_h (u - hn mean(u hn))        (the whole gradient of h)
//   dx = a D,  dg = D z,  q = g D v_out,  dy = r_y (q - yn mean(q yn)),
//   dv_in = sum over rows of dn hn,  dv_out = sum over rows of g D yn.
// A row stays in the registers of one workgroup from its load to its store, so every
// tensor crosses memory once.
#include <cfloat>
#include <cmath>

#include "rows.hpp"

namespace moe {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxThreads = 1024;

struct NormDev {
  const void *x, *y, *v_out, *v_in, *gate;
  int64_t x_stride, y_stride, gate_stride;
  int gate_kind, T, d;
  float scale, eps;
  // forward
  void *h, *n;
  int64_t h_stride, n_stride;
  // gradient
  const void *dh, *dn;
  void *dx, *dy, *dgate;
  int64_t dh_stride, dn_stride, dx_stride, dy_stride, dgate_stride;
  float* part;  // [workgroup][2][d]: column sums for v_out and gate, and for v_in; or null
};

template <typename S>
__device__ __forceinline__ const S* row_ptr(const void* p, int64_t t, int64_t stride) {
  return static_cast<const S*>(p) + t * stride;
}
template <typename S>
__device__ __forceinline__ S* row_ptr(void* p, int64_t t, int64_t stride) {
  return static_cast<S*>(p) + t * stride;
}

// How the threads of a workgroup share rows: `slots` rows at a time, each by 1 << lt lanes of a wavefront or by `waves` whole wavefronts.
struct NormSplit {
  int lt, waves, slots, threads, pieces;
};

// sums over the threads of a row, in each of them.  Rows of several wavefronts meet in
// LDS; the caller alternates between two buffers, so that one barrier is enough: a
// wavefront that writes a buffer again has passed the barrier of the other one, which
// every wavefront reaches after it has read the first.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], const NormSplit& p, float* buf) {
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = lane_sum(v[i], p.lt);
  if (p.waves == 1) return;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) buf[wave * 8 + i] = v[i];
  __syncthreads();
  const int first = wave - wave % p.waves;
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = 0.f;
  for (int w = first; w < first + p.waves; ++w)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += buf[w * 8 + i];
}

// Which row and lane of it a thread is.
struct RowLane {
  int slot, lane, lanes;
};
// kSub: rows by parts of wavefronts; else a wavefront has one row, whose number and
// addresses stay in scalar registers.
template <bool kSub>
__device__ __forceinline__ RowLane row_lane(const NormSplit& p) {
  if (kSub) return {(int)threadIdx.x >> p.lt, (int)threadIdx.x & ((1 << p.lt) - 1), 1 << p.lt};
  const int slot = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / p.waves);
  return {slot, (int)threadIdx.x - slot * p.waves * 64, p.waves * 64};
}

template <typename S>
__device__ __forceinline__ Raw<S> ones() {
  float v[kPiece];
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = 1.f;
  return pack<S>(v);
}

template <typename S>
__device__ __forceinline__ Raw<S> masked(Raw<S> r, uint32_t mask) {
#pragma unroll
  for (int q = 0; q < (int)(sizeof(r.w) / sizeof(r.w[0])); ++q) r.w[q] &= mask;
  return r;
}

template <typename S, int R, bool kSub>
__global__ __launch_bounds__(kNormMaxThreads) void k_block_norm(NormDev a, NormSplit p) {
  __shared__ float lds[2][kNormMaxThreads / 64 * 8];
  const RowLane rl = row_lane<kSub>(p);
  const int64_t t = (int64_t)blockIdx.x * p.slots + rl.slot;
  const bool live = t < a.T;
  const int64_t tc = live ? t : a.T - 1;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL, full = a.gate_kind == MOE_GATE_FULL;
  float h[R][kPiece], z[R][kPiece];
  Piece c[R];
  Raw<S> vo[R], vi[R], vg[R];
  float ss[1] = {0.f};
  // every load of the row before its first use
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = piece_of((r * rl.lanes + rl.lane) * kPiece, a.d);
    if (!live) c[r].skip = kPiece;
    const Raw<S> x = load_raw<kSub>(row_ptr<S>(a.x, tc, a.x_stride), c[r], a.d);
    unpack<S>(x, h[r]);
    if (a.y) load_piece<kSub>(row_ptr<S>(a.y, tc, a.y_stride), c[r], a.d, z[r]);
    vo[r] = vg[r] = vi[r] = ones<S>();
    if (a.v_out) vo[r] = load_raw<kSub>(static_cast<const S*>(a.v_out), c[r], a.d);
    if (channel || full)
      vg[r] = load_raw<kSub>(full ? row_ptr<S>(a.gate, tc, a.gate_stride) : static_cast<const S*>(a.gate), c[r], a.d);
    if (a.v_in) vi[r] = load_raw<kSub>(static_cast<const S*>(a.v_in), c[r], a.d);
  }
  const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(*row_ptr<S>(a.gate, tc, a.gate_stride)) : 1.f;
  float hh[1] = {0.f};
  if (a.y) {
    float ry = 1.f;
    if (a.v_out) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) ss[0] = fmaf(z[r][i], z[r][i], ss[0]);
      row_sums(ss, p, lds[0]);
      ry = rsqrtf(ss[0] / a.d + a.eps);
    }
    ry *= gt;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[kPiece], g[kPiece];
      unpack<S>(vo[r], v);
      unpack<S>(vg[r], g);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) h[r][i] = fmaf(ry * z[r][i], v[i] * g[i], a.scale * h[r][i]);
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) h[r][i] *= a.scale;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (a.h) store_piece<kSub>(row_ptr<S>(a.h, tc, a.h_stride), c[r], a.d, h[r]);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) hh[0] = fmaf(h[r][i], h[r][i], hh[0]);
  }
  if (!a.v_in) return;
  row_sums(hh, p, lds[1]);
  const float rh = rsqrtf(hh[0] / a.d + a.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v[kPiece];
    unpack<S>(vi[r], v);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] *= rh * h[r][i];
    store_piece<kSub>(row_ptr<S>(a.n, tc, a.n_stride), c[r], a.d, v);
  }
}

// The rows of the gradient, in registers: what the next row needs is requested before
// the arithmetic of the current one.  D = dh + r_h (u - mean(u hn) r_h h) is linear in
// dh, u and h, and with q = g v_out y (g the channel or full gate) the sum over q D that
// dy and a token's gate need is the same combination of the sums over q dh, q u and q h:
// so a row takes two rounds of sums (y^2, then the other
// five) and not four, each of which would wait for the one before.
// Column sums: only A = sum over rows of D yn (g D yn for a token's or full gate) and
// B = that of dn hn are kept; dnorm_out and a channel gate's gradient are A times the
// channel gate and v_out.
// What a call leaves out is read from a tensor that it has and masked to zero (v_out and
// the channel gate: ones), so that no load sits under a branch; only a full gate, a
// fifth stream, has a kernel of its own.
template <typename S, int R, int kThreads, bool kSub, bool kFull>
__global__ __launch_bounds__(kThreads, kThreads == 512 && R == 1 ? 4 : 1) void k_block_norm_backward(NormDev a,
                                                                                                      NormSplit p) {
  __shared__ float lds[kThreads * kPiece];
  const RowLane rl = row_lane<kSub>(p);
  const void* dh_in = a.dh ? a.dh : a.dn;
  const void* dn_in = a.dn ? a.dn : a.dh;
  const void* x_in = a.dn ? a.x : dh_in;
  const void* y_in = a.y ? a.y : x_in;
  const int64_t dh_ld = a.dh ? a.dh_stride : a.dn_stride, dn_ld = a.dn ? a.dn_stride : a.dh_stride;
  const int64_t x_ld = a.dn ? a.x_stride : dh_ld, y_ld = a.y ? a.y_stride : x_ld;
  const uint32_t dh_on = a.dh ? ~0u : 0u, dn_on = a.dn ? ~0u : 0u, y_on = a.y ? ~0u : 0u;
  float A[R][kPiece], B[R][kPiece];
  float W[R][kPiece], V[R][kPiece];  // v_out times the channel gate; v_in
  Piece c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = piece_of((r * rl.lanes + rl.lane) * kPiece, a.d);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      A[r][i] = B[r][i] = 0.f;
      W[r][i] = V[r][i] = 1.f;
    }
    if (a.v_out) load_piece<kSub>(static_cast<const S*>(a.v_out), c[r], a.d, W[r]);
    if (a.v_in) load_piece<kSub>(static_cast<const S*>(a.v_in), c[r], a.d, V[r]);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      float g[kPiece];
      load_piece<kSub>(static_cast<const S*>(a.gate), c[r], a.d, g);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) W[r][i] *= g[i];
    }
  }
  Raw<S> rx[R], ry_[R], rh_[R], rn[R], rg[R];
  auto request = [&](int64_t t) {
    const int64_t tc = t < a.T ? t : a.T - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Piece q = c[r];
      if (t >= a.T) q.skip = kPiece;
      ry_[r] = load_raw<kSub>(row_ptr<S>(y_in, tc, y_ld), q, a.d);
      rx[r] = load_raw<kSub>(row_ptr<S>(x_in, tc, x_ld), q, a.d);
      rn[r] = load_raw<kSub>(row_ptr<S>(dn_in, tc, dn_ld), q, a.d);
      rh_[r] = load_raw<kSub>(row_ptr<S>(dh_in, tc, dh_ld), q, a.d);
      if (kFull) rg[r] = load_raw<kSub>(row_ptr<S>(a.gate, tc, a.gate_stride), q, a.d);
    }
  };
  const int64_t step = (int64_t)gridDim.x * p.slots;
  const int64_t rounds = (a.T + step - 1) / step;
  int64_t t = (int64_t)blockIdx.x * p.slots + rl.slot;
  request(t);
  for (int64_t it = 0; it < rounds; ++it, t += step) {
    const bool live = t < a.T;
    const int64_t tc = live ? t : a.T - 1;
    Raw<S> x[R], y[R], dh[R], dn[R], g[R];
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // y y; then h h, u h, q dh, q u, q h
    float f[kPiece], e[kPiece];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = masked<S>(rx[r], dn_on);
      y[r] = masked<S>(ry_[r], y_on);
      dh[r] = masked<S>(rh_[r], dh_on);
      dn[r] = masked<S>(rn[r], dn_on);
      if (kFull) g[r] = rg[r];
      unpack<S>(y[r], f);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) s[0] = fmaf(f[i], f[i], s[0]);
    }
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(*row_ptr<S>(a.gate, tc, a.gate_stride)) : 1.f;
    request(t + step);
    float ry = 1.f;
    if (a.v_out) {
      float sy[1] = {s[0]};
      row_sums(sy, p, lds);
      ry = rsqrtf(sy[0] / a.d + a.eps);
    }
    float h[R][kPiece], q[R][kPiece], u[R][kPiece], D[R][kPiece];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      unpack<S>(y[r], q[r]);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) q[r][i] *= W[r][i];
      if (kFull) {
        unpack<S>(g[r], e);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) q[r][i] *= e[i];
      }
      unpack<S>(x[r], h[r]);
      unpack<S>(dn[r], u[r]);
      unpack<S>(dh[r], D[r]);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        h[r][i] = fmaf(gt * ry, q[r][i], a.scale * h[r][i]);
        u[r][i] *= V[r][i];
        s[1] = fmaf(h[r][i], h[r][i], s[1]);
        s[2] = fmaf(u[r][i], h[r][i], s[2]);
        s[3] = fmaf(q[r][i], D[r][i], s[3]);
        s[4] = fmaf(q[r][i], u[r][i], s[4]);
        s[5] = fmaf(q[r][i], h[r][i], s[5]);
      }
    }
    float rh = 0.f, mh = 0.f, qD = 0.f;
    if (a.dn || a.y) {
      float sum[5] = {s[1], s[2], s[3], s[4], s[5]};
      row_sums(sum, p, lds + kThreads / 64 * 8);
      rh = a.dn ? rsqrtf(sum[0] / a.d + a.eps) : 0.f;
      mh = rh * (sum[1] / a.d);  // mean(u hn)
      qD = sum[2] + rh * (sum[3] - mh * (rh * sum[4]));
    }
    // mean(g v_out D yn).  (Factors 1 / rms go with the sum or the element that they
    // scale, one at a time: their cube leaves float32's range for rows of size 1e13.)
    const float my = a.v_out ? gt * (ry * (qD / a.d)) : 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && live && rl.lane == 0) static_cast<float*>(a.dgate)[t] = ry * qD;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Piece w = c[r];
      if (!live) w.skip = kPiece;
      unpack<S>(dn[r], f);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const float hn = rh * h[r][i];
        B[r][i] = fmaf(f[i], hn, B[r][i]);
        D[r][i] += rh * (u[r][i] - mh * hn);
        f[i] = a.scale * D[r][i];
      }
      if (a.dx) store_piece<kSub>(row_ptr<S>(a.dx, tc, a.dx_stride), w, a.d, f);
      if (!a.y) continue;
      unpack<S>(y[r], e);
      float k[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        f[i] = W[r][i] * D[r][i];  // without the full or the token's gate
        e[i] *= ry;
        k[i] = gt;
      }
      if (kFull) {
        if (a.dgate) {
          float o[kPiece];
#pragma unroll
          for (int i = 0; i < kPiece; ++i) o[i] = f[i] * e[i];
          store_piece<kSub>(row_ptr<S>(a.dgate, tc, a.dgate_stride), w, a.d, o);
        }
        unpack<S>(g[r], k);
      }
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        A[r][i] = fmaf(k[i] * D[r][i], e[i], A[r][i]);
        f[i] = ry * (k[i] * f[i] - my * e[i]);
      }
      if (a.dy) store_piece<kSub>(row_ptr<S>(a.dy, tc, a.dy_stride), w, a.d, f);
    }
  }
  if (!a.part) return;
  // the slots' column sums, in slot order
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.d;
  const int width = rl.lanes * kPiece;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i >= c[r].skip && (!kSub || c[r].at + i < a.d))
          lds[rl.slot * width + c[r].at + i - r * width] = k == 0 ? A[r][i] : B[r][i];
      __syncthreads();
      for (int j = threadIdx.x; j < width && r * width + j < a.d; j += blockDim.x) {
        float v = 0.f;
        for (int g = 0; g < p.slots; ++g) v += lds[g * width + j];
        out[k * (int64_t)a.d + r * width + j] = v;
      }
    }
}

// the [d] gradients: column sums over the workgroups, 32 columns of A (blockIdx.y = 0)
// or B by 32 rows of threads
template <typename S>
__global__ __launch_bounds__(1024) void k_norm_vectors(const float* part, int groups, NormDev a, float* dv_out,
                                                       float* dv_in, float* dgate) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.d)
    for (int g = row; g < groups; g += 256)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (g + 32 * i < groups) s[i] += part[((int64_t)(g + 32 * i) * 2 + blockIdx.y) * a.d + c];
  lds[row][x] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (row != 0 || c >= a.d) return;
  float v = 0.f;
  for (int r = 0; r < 32; ++r) v += lds[r][x];
  if (blockIdx.y == 1) {
    if (dv_in) dv_in[c] = v;
    return;
  }
  if (dgate) dgate[c] = a.v_out ? v * to_f32(static_cast<const S*>(a.v_out)[c]) : v;
  if (dv_out) dv_out[c] = a.gate_kind == MOE_GATE_CHANNEL ? v * to_f32(static_cast<const S*>(a.gate)[c]) : v;
}

// `target` threads per workgroup, more where one row needs them
static NormSplit norm_split(int d, int target) {
  NormSplit p;
  const int pieces = (int)ceil_div(d, kPiece);
  p.pieces = pieces <= 512 ? 1 : 2;
  const int lanes = (int)ceil_div(pieces, p.pieces);
  p.lt = 0;
  while (p.lt < 6 && (1 << p.lt) < lanes) ++p.lt;
  p.waves = (int)ceil_div(lanes, 64);
  p.slots = p.waves > 1 ? std::max(1, target / (64 * p.waves)) : target >> p.lt;
  p.threads = p.waves > 1 ? p.slots * 64 * p.waves : target;
  return p;
}

// workgroups of the gradient: two per CU, few enough that their column sums stay small
// beside the rows
static int norm_groups(int T, int d) {
  return (int)std::min<int64_t>(ceil_div(T, norm_split(d, 512).slots), 512);
}

static int check_norm(const char* fn, const moe_block_norm_args* a) {
  MOE_CHECK_ARG(a != nullptr, MOE_ERR_INVALID_ARG, "%s: args is NULL", fn);
  MOE_CHECK_ARG(a->dtype >= MOE_BF16 && a->dtype <= MOE_FP32, MOE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, a->dtype);
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0, MOE_ERR_INVALID_ARG, "%s: bad sizes T=%d d=%d", fn, a->T, a->d);
  MOE_CHECK_ARG(a->d <= kNormMaxD && a->T <= (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: unsupported T=%d d=%d (T <= 2^24, d <= %d)", fn, a->T, a->d, kNormMaxD);
  MOE_CHECK_ARG(a->gate_kind >= MOE_GATE_NONE && a->gate_kind <= MOE_GATE_FULL, MOE_ERR_INVALID_ARG,
                "%s: bad gate_kind %d", fn, a->gate_kind);
  MOE_CHECK_ARG(a->eps >= FLT_MIN && std::isfinite(a->eps) && std::isfinite(a->residual_scale), MOE_ERR_INVALID_ARG,
                "%s: eps %g or residual_scale %g out of range", fn, (double)a->eps, (double)a->residual_scale);
  const int64_t size = dtype_bytes(a->dtype);
  for (const void* p : {a->x, a->y, a->norm_out, a->norm_in, a->gate})
    MOE_CHECK_ARG(((uintptr_t)p % size) == 0, MOE_ERR_INVALID_ARG, "%s: misaligned input", fn);
  if (a->T == 0) return MOE_OK;  // no rows: their pointers may be NULL
  MOE_CHECK_ARG(a->x, MOE_ERR_INVALID_ARG, "%s: x is NULL", fn);
  MOE_CHECK_ARG(a->y || (!a->norm_out && a->gate_kind == MOE_GATE_NONE), MOE_ERR_INVALID_ARG,
                "%s: norm_out and gate need y", fn);
  MOE_CHECK_ARG((a->gate != nullptr) == (a->gate_kind != MOE_GATE_NONE), MOE_ERR_INVALID_ARG,
                "%s: gate and gate_kind %d disagree", fn, a->gate_kind);
  MOE_CHECK_ARG(a->x_stride >= 0 && (!a->y || a->y_stride >= 0) &&
                    (a->gate_kind < MOE_GATE_TOKEN || a->gate_stride >= 0),
                MOE_ERR_INVALID_ARG, "%s: negative stride", fn);
  return MOE_OK;
}

static int check_row_tensor(const char* fn, const char* name, const void* p, int64_t stride, int64_t least,
                            int64_t size) {
  MOE_CHECK_ARG(!p || (((uintptr_t)p % size) == 0 && stride >= least), MOE_ERR_INVALID_ARG,
                "%s: %s misaligned or stride %lld below %lld", fn, name, (long long)stride, (long long)least);
  return MOE_OK;
}

static NormDev norm_dev(const moe_block_norm_args* a) {
  NormDev v{};
  v.x = a->x;
  v.y = a->y;
  v.v_out = a->norm_out;
  v.v_in = a->norm_in;
  v.gate = a->gate;
  v.x_stride = a->x_stride;
  v.y_stride = a->y_stride;
  v.gate_stride = a->gate_stride;
  v.gate_kind = a->gate_kind;
  v.T = a->T;
  v.d = a->d;
  v.scale = a->residual_scale;
  v.eps = a->eps;
  return v;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_block_norm(const moe_block_norm_args* a, void* h, int64_t h_stride, void* n, int64_t n_stride,
                              void* stream) {
  clear_error();
  const char* fn = "moe_block_norm";
  int rc = check_norm(fn, a);
  if (rc) return rc;
  if (a->T == 0) return MOE_OK;
  const int64_t size = dtype_bytes(a->dtype);
  MOE_CHECK_ARG(h || n, MOE_ERR_INVALID_ARG, "%s: neither h nor n is wanted", fn);
  MOE_CHECK_ARG((n != nullptr) == (a->norm_in != nullptr), MOE_ERR_INVALID_ARG, "%s: n goes with norm_in", fn);
  if ((rc = check_row_tensor(fn, "h", h, h_stride, a->d, size))) return rc;
  if ((rc = check_row_tensor(fn, "n", n, n_stride, a->d, size))) return rc;
  NormDev v = norm_dev(a);
  v.h = h;
  v.h_stride = h_stride;
  v.n = n;
  v.n_stride = n_stride;
  hipStream_t s = (hipStream_t)stream;
  const NormSplit p = norm_split(a->d, 256);
  const dim3 grid((unsigned)ceil_div(a->T, p.slots));
  timing_begin(K_BLOCK_NORM, s);
  with_dtype(a->dtype, [&](auto e) {
    using S = decltype(e);
    if (p.lt < 6)
      hipLaunchKernelGGL((k_block_norm<S, 1, true>), grid, dim3(p.threads), 0, s, v, p);
    else if (p.pieces == 1)
      hipLaunchKernelGGL((k_block_norm<S, 1, false>), grid, dim3(p.threads), 0, s, v, p);
    else
      hipLaunchKernelGGL((k_block_norm<S, 2, false>), grid, dim3(p.threads), 0, s, v, p);
  });
  timing_end(K_BLOCK_NORM, s);
  return check_launch(fn);
}

extern "C" int64_t moe_block_norm_backward_workspace_bytes(int T, int d) {
  if (T < 0 || d <= 0) return -1;
  return (int64_t)norm_groups(T, d) * 2 * d * 4;
}

extern "C" int moe_block_norm_backward(const moe_block_norm_args* a, const moe_block_norm_grads* g, void* stream) {
  clear_error();
  const char* fn = "moe_block_norm_backward";
  int rc = check_norm(fn, a);
  if (rc) return rc;
  MOE_CHECK_ARG(g != nullptr, MOE_ERR_INVALID_ARG, "%s: grads is NULL", fn);
  const int64_t size = dtype_bytes(a->dtype);
  if ((rc = check_row_tensor(fn, "dh", g->dh, g->dh_stride, 0, size))) return rc;
  if ((rc = check_row_tensor(fn, "dn", g->dn, g->dn_stride, 0, size))) return rc;
  if ((rc = check_row_tensor(fn, "dx", g->dx, g->dx_stride, a->d, size))) return rc;
  if ((rc = check_row_tensor(fn, "dy", g->dy, g->dy_stride, a->d, size))) return rc;
  const bool full = a->gate_kind == MOE_GATE_FULL;
  if ((rc = check_row_tensor(fn, "dgate", g->dgate, full ? g->dgate_stride : 0, full ? a->d : 0, full ? size : 4)))
    return rc;
  if ((rc = check_row_tensor(fn, "dnorm_out", g->dnorm_out, 0, 0, 4))) return rc;
  if ((rc = check_row_tensor(fn, "dnorm_in", g->dnorm_in, 0, 0, 4))) return rc;
  MOE_CHECK_ARG(a->T == 0 || g->dh || g->dn, MOE_ERR_INVALID_ARG, "%s: neither dh nor dn is given", fn);
  MOE_CHECK_ARG((!g->dn || a->norm_in) && (!g->dnorm_in || a->norm_in), MOE_ERR_INVALID_ARG,
                "%s: dn and dnorm_in need norm_in", fn);
  MOE_CHECK_ARG((!g->dy || a->y) && (!g->dnorm_out || a->norm_out) &&
                    (!g->dgate || a->gate_kind != MOE_GATE_NONE),
                MOE_ERR_INVALID_ARG, "%s: dy, dnorm_out and dgate need y, norm_out and gate", fn);
  float* dgate_vec = a->gate_kind == MOE_GATE_CHANNEL ? static_cast<float*>(g->dgate) : nullptr;
  const bool vectors = g->dnorm_out || g->dnorm_in || dgate_vec;
  const int64_t need = moe_block_norm_backward_workspace_bytes(a->T, a->d);
  MOE_CHECK_ARG(!vectors || a->T == 0 ||
                    (g->workspace && g->workspace_bytes >= need && ((uintptr_t)g->workspace % 256) == 0),
                MOE_ERR_WORKSPACE, "%s: workspace of %lld bytes < %lld needed, NULL or misaligned", fn,
                (long long)g->workspace_bytes, (long long)need);
  if (a->T == 0 && !vectors) return MOE_OK;
  NormDev v = norm_dev(a);
  v.dh = g->dh;
  v.dh_stride = g->dh_stride;
  v.dn = g->dn;
  v.dn_stride = g->dn_stride;
  v.dx = g->dx;
  v.dx_stride = g->dx_stride;
  v.dy = g->dy;
  v.dy_stride = g->dy_stride;
  v.dgate = g->dgate;
  v.dgate_stride = g->dgate_stride;
  v.part = vectors ? static_cast<float*>(g->workspace) : nullptr;
  hipStream_t s = (hipStream_t)stream;
  const NormSplit p = norm_split(a->d, 512);
  const int groups = norm_groups(a->T, a->d);
  timing_begin(K_BLOCK_NORM_BWD, s);
  with_dtype(a->dtype, [&](auto e) {
    using S = decltype(e);
    if (a->T > 0) {
      auto go = [&](auto pieces, auto threads, auto sub) {
        constexpr int R = decltype(pieces)::value, B = decltype(threads)::value;
        constexpr bool kSub = decltype(sub)::value;
        if (a->gate_kind == MOE_GATE_FULL)
          hipLaunchKernelGGL((k_block_norm_backward<S, R, B, kSub, true>), dim3(groups), dim3(p.threads), 0, s, v, p);
        else
          hipLaunchKernelGGL((k_block_norm_backward<S, R, B, kSub, false>), dim3(groups), dim3(p.threads), 0, s, v, p);
      };
      using std::integral_constant;
      if (p.lt < 6)
        go(integral_constant<int, 1>{}, integral_constant<int, 512>{}, std::true_type{});
      else if (p.pieces == 1)
        go(integral_constant<int, 1>{}, integral_constant<int, 512>{}, std::false_type{});
      else if (p.threads <= 512)
        go(integral_constant<int, 2>{}, integral_constant<int, 512>{}, std::false_type{});
      else
        go(integral_constant<int, 2>{}, integral_constant<int, 1024>{}, std::false_type{});
    }
    if (vectors)
      hipLaunchKernelGGL(k_norm_vectors<S>, dim3((unsigned)ceil_div(a->d, 32), 2), dim3(1024), 0, s, v.part, groups, v,
                         g->dnorm_out, g->dnorm_in, dgate_vec);
  });
  timing_end(K_BLOCK_NORM_BWD, s);
  return check_launch(fn);
}

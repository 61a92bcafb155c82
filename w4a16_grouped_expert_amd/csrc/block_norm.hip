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
// A row stays in the registers of its wavefronts from its load to its store, so every
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
  float scale, eps, inv_d;
  // forward
  void *h, *n;
  int64_t h_stride, n_stride;
  // gradient
  const void *dh, *dn;
  void *dx, *dy, *dgate;
  int64_t dh_stride, dn_stride, dx_stride, dy_stride, dgate_stride;
  float* part;  // [workgroup][2][d]: column sums for v_out and gate, and for v_in; or null
  float *dv_out, *dv_in, *dgate_vec;  // the [d] gradients, null where not wanted
};

template <typename S, bool kSub>
__device__ __forceinline__ float token_gate(const NormDev& a, int64_t t) {
  return a.gate_kind == MOE_GATE_TOKEN ? load_one(row_ptr<S, kSub>(a.gate, t, a.gate_stride)) : 1.f;
}

// How the threads of a workgroup share rows: `slots` rows at a time, each by 1 << lt
// lanes of a wavefront or by `waves` whole wavefronts.
struct NormSplit {
  int lt, waves, slots, threads, pieces;
};

// The same value, unknown to the compiler and settled here: nothing that depends on it is
// kept from before, moved out of a loop, or put off until later.
template <typename V>
__device__ __forceinline__ void forget(V& v) {
  asm volatile("" : "+v"(v));
}
template <typename S>
__device__ __forceinline__ void forget(Raw<S>& r) {
#pragma unroll
  for (int q = 0; q < (int)(sizeof(r.w) / sizeof(r.w[0])); ++q) asm volatile("" : "+v"(r.w[q]) : : "memory");
}

// sums over the threads of a row, in each of them.  Rows of several wavefronts meet in
// LDS.  One call after the other takes the other of two buffers (the caller counts them),
// so that one barrier is enough: a wavefront that writes a buffer again has passed the
// barrier of the other one, which every wavefront reaches after it has read the first.
template <bool kSub, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], const NormSplit& p, float* buf) {
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = lane_sum(v[i], kSub ? p.lt : 6);
  if (kSub || p.waves == 1) return;
  int tid = threadIdx.x;
  forget(tid);  // (addresses made from it outside the caller's loop would stay in registers)
  const int wave = tid >> 6;
  if ((tid & 63) == 0)
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

// a piece's own elements, zero for those of the piece before
template <typename S>
__device__ __forceinline__ void unpack_own(Raw<S> r, Piece p, float (&v)[kPiece]) {
  forget(p.skip);  // (or its masks would stay in registers through the caller's loop)
  mask_piece(r, p);
  unpack<S>(r, v);
}

// Forward: a row by as many lanes as it has pieces, up to 512 of them; longer rows two
// pieces per lane.  Bound by HBM: T = 16384, d = 2048 in bf16, x and y read, h and n
// written, 268 MB in 48 us (5.6 TB/s); 16 rows take 3.6 us, a launch and the row's chain of
// loads and two sums.
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
  Raw<S> rx[R], ry_[R], vo[R], vi[R], vg[R];
  float ss[1] = {0.f};
  // every load of the row before its first use
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = piece_of((r * rl.lanes + rl.lane) * kPiece, a.d);
    rx[r] = load_raw<kSub>(row_ptr<S, kSub>(a.x, tc, a.x_stride), c[r], a.d);
    if (a.y) ry_[r] = load_raw<kSub>(row_ptr<S, kSub>(a.y, tc, a.y_stride), c[r], a.d);
    vo[r] = vg[r] = vi[r] = ones<S>();
    if (a.v_out) vo[r] = load_raw<kSub>(static_cast<const S*>(a.v_out), c[r], a.d);
    if (channel || full)
      vg[r] = load_raw<kSub>(full ? row_ptr<S, kSub>(a.gate, tc, a.gate_stride) : static_cast<const S*>(a.gate), c[r], a.d);
    if (a.v_in) vi[r] = load_raw<kSub>(static_cast<const S*>(a.v_in), c[r], a.d);
  }
  const float gt = token_gate<S, kSub>(a, tc);
  // (x and y are in registers before the barrier that the first store waits for: h may lie
  // where they do, and the last pieces of two wavefronts may overlap)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    forget(rx[r]);
    unpack<S>(rx[r], h[r]);
    if (a.y) {
      forget(ry_[r]);
      unpack<S>(ry_[r], z[r]);
    }
  }
  float hh[1] = {0.f};
  if (a.y) {
    float ry = 1.f;
    if (a.v_out) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) ss[0] = i < c[r].skip ? ss[0] : fmaf(z[r][i], z[r][i], ss[0]);
      row_sums<kSub>(ss, p, lds[0]);
      ry = rsqrtf(ss[0] * a.inv_d + a.eps);
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
  if (!kSub && p.waves > 1 && !a.v_out) __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (a.h && live) store_piece<kSub>(row_ptr<S, kSub>(a.h, tc, a.h_stride), c[r], a.d, h[r]);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) hh[0] = i < c[r].skip ? hh[0] : fmaf(h[r][i], h[r][i], hh[0]);
  }
  if (!a.v_in) return;
  row_sums<kSub>(hh, p, lds[1]);
  const float rh = rsqrtf(hh[0] * a.inv_d + a.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v[kPiece];
    unpack<S>(vi[r], v);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] *= rh * h[r][i];
    if (live) store_piece<kSub>(row_ptr<S, kSub>(a.n, tc, a.n_stride), c[r], a.d, v);
  }
}

// a piece of `out` (null: not wanted) = v times that of `factor` (null: 1)
template <bool kSub, typename S>
__device__ __forceinline__ void store_times(float* out, const S* factor, const Piece& c, int d, const float (&v)[kPiece]) {
  if (!out) return;
  float f[kPiece];
#pragma unroll
  for (int i = 0; i < kPiece; ++i) f[i] = 1.f;
  if (factor) unpack<S>(load_raw<kSub>(factor, c, d), f);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) f[i] = factor ? v[i] * f[i] : v[i];
  store_piece<kSub, false>(out, c, d, f);
}

// The gradient.  D = dh + r_h (u - mean(u hn) r_h h) is linear in dh, u and h, and with
// q = g v_out y (g the channel or full gate) the sum over q D that dy and a token's gate
// need is the same combination of the sums over q dh, q u and q h: so a row takes two
// rounds of sums (y^2, then the other five) and not four, each of which would wait for
// the one before.
//
// A row belongs to one wavefront where R pieces per lane hold it, so that its
// sums need no barrier and the wavefronts of a CU drift apart: some load while others
// compute.  Only the row as loaded and the column sums stay in registers; h, u and q are
// computed again for the outputs, one piece after the other, v_out times the channel gate
// (W) and v_in (V) come from LDS.  The forget() calls hold the compiler to that: left
// alone it keeps every piece's floats, 3 x 8 R registers, and spills.
// Column sums: only A = sum over rows of D yn (g D yn for a token's or full gate) and
// B = that of dn hn are kept; dnorm_out and a channel gate's gradient are A times the
// channel gate and v_out.
// Measured: T = 8192, d = 2048 in bf16 42 us for 201 MB (4.7 TB/s) and 5 for the sums
// over the workgroups, with a full gate 56 us for 268 MB (4.8 TB/s); 1001 rows of 1111 floats
// 11.0 and 4.4 us; 4096 rows of 1280 floats with a full gate 38 us for 168 MB (4.4 TB/s).
// Many rows are bound by HBM and the launch around them; few rows by the chain of one row,
// some 6 us from the first load to the column sums, and the two launches.  Two
// wavefronts per SIMD that request x and y of the next row ran faster than one that requests all of it
// (46.9 to 45.2 us for both launches) or two that request nothing (46.2); dn and dh requested
// early too, or column sums that all slots hand over at once, changed nothing.
// What a call leaves out is read from a tensor that it has and masked to zero, so that no
// load sits under a branch; only a full gate, a fifth stream, has a kernel of its own.
//
// Wavefronts per workgroup, one workgroup per CU: what the registers of a row of `bytes`
// per element and R pieces allow.
constexpr int norm_back_waves(int R, int bytes) { return R == 1 ? 16 : R == 2 && bytes == 2 ? 12 : 8; }

template <typename S, int R, bool kSub, bool kFull>
__global__ __launch_bounds__(64 * norm_back_waves(R, sizeof(S))) void k_block_norm_backward(NormDev a, NormSplit p) {
  __shared__ float sums[2][16 * 8];
  // [wavefront of the row][W, V][R][half][lane]: four elements of a lane's piece each
  extern __shared__ f32x4_t vec[];
  const RowLane rl = row_lane<kSub>(p);
  const void* dh_in = a.dh ? a.dh : a.dn;
  const void* dn_in = a.dn ? a.dn : a.dh;
  const void* x_in = a.dn ? a.x : dh_in;
  const void* y_in = a.y ? a.y : x_in;
  const int64_t dh_ld = a.dh ? a.dh_stride : a.dn_stride, dn_ld = a.dn ? a.dn_stride : a.dh_stride;
  const int64_t x_ld = a.dn ? a.x_stride : dh_ld, y_ld = a.y ? a.y_stride : x_ld;
  const uint32_t dh_on = __builtin_amdgcn_readfirstlane(a.dh ? ~0u : 0u);
  const uint32_t dn_on = __builtin_amdgcn_readfirstlane(a.dn ? ~0u : 0u);
  const uint32_t y_on = __builtin_amdgcn_readfirstlane(a.y ? ~0u : 0u);
  float A[R][kPiece], B[R][kPiece];
  int turn = 0;  // of the sums' buffers: a row without norm_out has one round of sums, others two
  Piece c[R];
  f32x4_t* const vec_mine = vec + (rl.lane >> 6) * (4 * R * 64) + (rl.lane & 63);
  auto vec_at = [&](int k, int r, int half) -> f32x4_t& { return vec_mine[((k * R + r) * 2 + half) * 64]; };
  auto vec_put = [&](int k, int r, const float (&v)[kPiece]) {
    vec_at(k, r, 0) = f32x4_t{v[0], v[1], v[2], v[3]};
    vec_at(k, r, 1) = f32x4_t{v[4], v[5], v[6], v[7]};
  };
  auto vec_get = [&](int k, int r, float (&v)[kPiece]) {
    const f32x4_t lo = vec_at(k, r, 0), hi = vec_at(k, r, 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = lo[i];
      v[4 + i] = hi[i];
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = piece_of((r * rl.lanes + rl.lane) * kPiece, a.d);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) A[r][i] = B[r][i] = 0.f;
  }
  if (rl.slot == 0) {
    // (every load before the first use: what is missing is read from x and replaced)
    const S* any = static_cast<const S*>(a.x);
    const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
    Raw<S> vo[R], vi[R], vg[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      vo[r] = load_raw<kSub>(a.v_out ? static_cast<const S*>(a.v_out) : any, c[r], a.d);
      vi[r] = load_raw<kSub>(a.v_in ? static_cast<const S*>(a.v_in) : any, c[r], a.d);
      vg[r] = load_raw<kSub>(channel ? static_cast<const S*>(a.gate) : any, c[r], a.d);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[kPiece], w[kPiece], g[kPiece];
      unpack<S>(vo[r], w);
      unpack<S>(vi[r], v);
      unpack<S>(vg[r], g);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        w[i] = (a.v_out ? w[i] : 1.f) * (channel ? g[i] : 1.f);
        v[i] = a.v_in ? v[i] : 1.f;
      }
      vec_put(0, r, w);
      vec_put(1, r, v);
    }
  }
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * p.slots;
  const int64_t rounds = (a.T + step - 1) / step;
  int64_t t = (int64_t)blockIdx.x * p.slots + rl.slot;
  // y and x of the next row are requested before the arithmetic of the current one, dn and
  // dh at its start: what the registers allow at two wavefronts per SIMD
  Raw<S> next_x[R], next_y[R];
  auto request = [&](int64_t t) {
#pragma unroll
    for (int r = 0; r < R; ++r) next_y[r] = load_raw<kSub>(row_ptr<S, kSub>(y_in, t, y_ld), c[r], a.d);
#pragma unroll
    for (int r = 0; r < R; ++r) next_x[r] = load_raw<kSub>(row_ptr<S, kSub>(x_in, t, x_ld), c[r], a.d);
  };
  request(t < a.T ? t : a.T - 1);
  for (int64_t it = 0; it < rounds; ++it, t += step) {
    const bool live = t < a.T;
    const int64_t tc = live ? t : a.T - 1;
    Raw<S> x[R], y[R], dh[R], dn[R], g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      dn[r] = load_raw<kSub>(row_ptr<S, kSub>(dn_in, tc, dn_ld), c[r], a.d);
      dh[r] = load_raw<kSub>(row_ptr<S, kSub>(dh_in, tc, dh_ld), c[r], a.d);
      if (kFull) g[r] = load_raw<kSub>(row_ptr<S, kSub>(a.gate, tc, a.gate_stride), c[r], a.d);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = next_x[r];
      y[r] = next_y[r];
      forget(x[r]);
      forget(y[r]);
    }
    if (t + step < a.T) request(t + step);
    const float gt = token_gate<S, kSub>(a, tc);
    float sy[1] = {0.f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      y[r] = masked<S>(y[r], y_on);
      float f[kPiece];
      unpack_own(y[r], c[r], f);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sy[0] = fmaf(f[i], f[i], sy[0]);
    }
    float ry = 1.f;
    if (a.v_out) {
      row_sums<kSub>(sy, p, sums[turn]);
      turn ^= 1;
      ry = rsqrtf(sy[0] * a.inv_d + a.eps);
    }
    // the piece's u, q and h, scaled: sx x + sq q
    auto piece = [&](int r, float sx, float sq, float (&h)[kPiece], float (&u)[kPiece], float (&q)[kPiece]) {
      float w[kPiece];
      unpack<S>(y[r], q);
      vec_get(0, r, w);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) q[i] *= w[i];
      if (kFull) {
        unpack<S>(g[r], w);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) q[i] *= w[i];
      }
      unpack<S>(x[r], h);
      unpack<S>(dn[r], u);
      vec_get(1, r, w);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        h[i] = fmaf(sq, q[i], sx * h[i]);
        u[i] *= w[i];
      }
    };
    float s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // h h, u h, q dh, q u, q h
#pragma unroll
    for (int r = 0; r < R; ++r) {
      forget(y[r]);
      forget(x[r]);
      forget(dn[r]);
      forget(dh[r]);
      x[r] = masked<S>(x[r], dn_on);
      dn[r] = masked<S>(dn[r], dn_on);
      dh[r] = masked<S>(dh[r], dh_on);
      float h[kPiece], u[kPiece], q[kPiece], D[kPiece];
      piece(r, a.scale, gt * ry, h, u, q);
      unpack<S>(dh[r], D);
      // Elements of the piece before are in its sums.  Here every factor of their products is
      // cleared (an infinite one times zero would be NaN), by a branch that few wavefronts take,
      // or each term left out where floats fill the registers: the one costs floats with a full
      // gate 6 % (T = 4096, d = 1280 44.4 to 47.1 us, left out 41.2), the other two bytes 4 %
      // (T = 3000, d = 1111 19.9 to 20.7, cleared 20.1).
      int skip = c[r].skip;
      forget(skip);
      constexpr bool kClear = sizeof(S) == 2;
      if (kClear && skip) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          h[i] = i < skip ? 0.f : h[i];
          u[i] = i < skip ? 0.f : u[i];
          q[i] = i < skip ? 0.f : q[i];
          D[i] = i < skip ? 0.f : D[i];
        }
      }
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        if (!kClear && i < skip) continue;
        s[0] = fmaf(h[i], h[i], s[0]);
        s[1] = fmaf(u[i], h[i], s[1]);
        s[2] = fmaf(q[i], D[i], s[2]);
        s[3] = fmaf(q[i], u[i], s[3]);
        s[4] = fmaf(q[i], h[i], s[4]);
      }
#pragma unroll
      for (int i = 0; i < 5; ++i) forget(s[i]);
    }
    row_sums<kSub>(s, p, sums[turn]);  // (its barrier also ends the row's loads before a store in their place)
    turn ^= 1;
    const float rh = a.dn ? rsqrtf(s[0] * a.inv_d + a.eps) : 0.f;
    // (without dn neither h nor its sums are used: y, and so h, may be infinite)
    const float mh = a.dn ? rh * (s[1] * a.inv_d) : 0.f;  // mean(u hn)
    const float qD = a.dn ? s[2] + rh * (s[3] - mh * (rh * s[4])) : s[2];
    // mean(g v_out D yn).  (Factors 1 / rms go with the sum or the element that they
    // scale, one at a time: their cube leaves float32's range for rows of size 1e13.)
    const float my = a.v_out ? gt * (ry * (qD * a.inv_d)) : 0.f;
    if (!live) continue;  // (a row past the last took part in the barriers, on the last row's values)
    if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && rl.lane == 0) static_cast<float*>(a.dgate)[t] = ry * qD;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      forget(y[r]);
      forget(x[r]);
      forget(dn[r]);
      forget(dh[r]);
      if (kFull) forget(g[r]);
      float h[kPiece], u[kPiece], D[kPiece], f[kPiece], e[kPiece];
      unpack<S>(dh[r], D);
      if (a.dn) {
        piece(r, rh * a.scale, rh * (gt * ry), h, u, f);  // hn in place of h
        unpack<S>(dn[r], f);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          B[r][i] = fmaf(f[i], h[i], B[r][i]);
          D[i] = fmaf(-rh * mh, h[i], fmaf(rh, u[i], D[i]));
          forget(B[r][i]);  // (put off, the addition would keep its operands to the end of the row)
        }
      }
#pragma unroll
      for (int i = 0; i < kPiece; ++i) f[i] = a.scale * D[i];
      if (a.dx) store_piece<kSub>(row_ptr<S, kSub>(a.dx, tc, a.dx_stride), c[r], a.d, f);
      if (a.y) {
        unpack<S>(y[r], e);
        vec_get(0, r, u);
        if (kFull) {
          float k[kPiece];
          unpack<S>(g[r], k);
#pragma unroll
          for (int i = 0; i < kPiece; ++i) {
            e[i] *= ry;
            f[i] = D[i] * (u[i] * e[i]);
            D[i] *= k[i];
          }
          if (a.dgate) store_piece<kSub>(row_ptr<S, kSub>(a.dgate, tc, a.dgate_stride), c[r], a.d, f);
        } else {
#pragma unroll
          for (int i = 0; i < kPiece; ++i) {
            e[i] *= ry;
            D[i] *= gt;
          }
        }
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          A[r][i] = fmaf(D[i], e[i], A[r][i]);
          f[i] = ry * (u[i] * D[i]);
          if (a.v_out) f[i] = fmaf(-ry * my, e[i], f[i]);  // (without norm_out y may be infinite)
          forget(A[r][i]);
        }
        if (a.dy) store_piece<kSub>(row_ptr<S, kSub>(a.dy, tc, a.dy_stride), c[r], a.d, f);
      }
    }
  }
  if (!a.part) return;
  // The slots' column sums, pairwise: the upper half of the slots hands its sums to the
  // lower one, until one slot has them.
  const int pitch = (p.slots / 2) * rl.lanes;  // threads that hand over in the first round
  auto hand_at = [&](int k, int slot) -> f32x4_t& { return vec[k * pitch + slot * rl.lanes + rl.lane]; };
  for (int n = p.slots; n > 1;) {
    const int half = (n + 1) / 2;
    __syncthreads();
    if (rl.slot >= half && rl.slot < n) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          hand_at(4 * r + k, rl.slot - half) =
              f32x4_t{A[r][4 * k], A[r][4 * k + 1], A[r][4 * k + 2], A[r][4 * k + 3]};
          hand_at(4 * r + 2 + k, rl.slot - half) =
              f32x4_t{B[r][4 * k], B[r][4 * k + 1], B[r][4 * k + 2], B[r][4 * k + 3]};
        }
    }
    __syncthreads();
    if (rl.slot < n - half) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const f32x4_t u = hand_at(4 * r + k, rl.slot), v = hand_at(4 * r + 2 + k, rl.slot);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            A[r][4 * k + i] += u[i];
            B[r][4 * k + i] += v[i];
          }
        }
    }
    n = half;
  }
  if (rl.slot != 0) return;
  if (gridDim.x == 1) {  // every row was this workgroup's
    const S* gate = a.gate_kind == MOE_GATE_CHANNEL ? static_cast<const S*>(a.gate) : nullptr;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (a.dv_in) store_piece<kSub, false>(a.dv_in, c[r], a.d, B[r]);
      store_times<kSub>(a.dgate_vec, static_cast<const S*>(a.v_out), c[r], a.d, A[r]);
      store_times<kSub>(a.dv_out, gate, c[r], a.d, A[r]);
    }
    return;
  }
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    store_piece<kSub, false>(out, c[r], a.d, A[r]);
    store_piece<kSub, false>(out + a.d, c[r], a.d, B[r]);
  }
}

// the [d] gradients: column sums over the workgroups, 32 columns of A (blockIdx.y = 0)
// or B by 32 rows of threads, each with eight loads in flight; 5 us for 256 workgroups
// of 2048 columns (4 MB), its launch and two dependent steps
template <typename S>
__global__ __launch_bounds__(1024) void k_norm_vectors(const float* part, int groups, NormDev a) {
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
    if (a.dv_in) a.dv_in[c] = v;
    return;
  }
  // (without rows the sums are zero, whatever the vectors hold)
  if (a.dgate_vec) a.dgate_vec[c] = a.v_out && groups ? v * load_one(static_cast<const S*>(a.v_out) + c) : v;
  if (a.dv_out)
    a.dv_out[c] = a.gate_kind == MOE_GATE_CHANNEL && groups ? v * load_one(static_cast<const S*>(a.gate) + c) : v;
}

// Forward: `target` threads per workgroup, more where one row needs them.
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

// Gradient: the pieces per lane (one to four) with which a workgroup has the most rows at
// once; among equals a row of one wavefront, which needs no barrier, then the fewest pieces
// per lane, that is the most wavefronts.  So rows of up to 2048 elements of two bytes or 1536
// floats have one wavefront.  (bf16: d = 2560 three pieces 34.7 us, four 38.6; 5120 two
// 46.8, four 52.7; 4096 four 49.4, two 51.1; 8192 four 50.4, two 54.3.)  Four pieces of floats
// spill some 100 registers, 180 with a full gate: only rows that nothing else takes have them.
// (Of the others, floats with a full gate spill one register in rows by parts of a wavefront
// and two with three pieces.)
static NormSplit norm_back_split(int T, int d, int dtype) {
  NormSplit p;
  const int bytes = (int)dtype_bytes(dtype);
  const int pieces = (int)ceil_div(d, kPiece);
  int rows = 0;
  for (int R = 1; R <= 4; ++R) {
    const int waves = (int)ceil_div(pieces, 64 * R), slots = norm_back_waves(R, bytes) / waves;
    if (R == 4 && bytes == 4 && rows > 0) continue;
    if (slots > rows || (slots == rows && slots > 0 && waves == 1 && p.waves > 1)) {
      rows = slots;
      p.pieces = R;
      p.waves = waves;
    }
  }
  const int lanes = (int)ceil_div(pieces, p.pieces);
  p.lt = 0;
  while (p.lt < 6 && (1 << p.lt) < lanes) ++p.lt;
  const int most = norm_back_waves(p.pieces, bytes);
  const int per_wave = 64 >> p.lt;
  int groups = p.waves > 1 ? most / p.waves : most;  // wavefronts (or groups of them) per workgroup
  // as many rows as a workgroup takes at once are its own, without a launch for the column
  // sums (calls of one row of 2048 bf16 12.1 to 9.0 us, of eight 11.9 to 11.0)
  const bool one = T <= groups * per_wave;
  // otherwise as many as its share of rows takes in as few rounds (fp16, T = 3894, d = 704: two
  // rounds of 8 rows 17.1 us, of 12 and 4 20.2)
  const int64_t share = ceil_div(T, one ? 1 : 256), rounds = std::max<int64_t>(1, ceil_div(share, groups * per_wave));
  groups = (int)std::max<int64_t>(1, ceil_div(share, per_wave * rounds));
  p.slots = groups * per_wave;
  p.threads = groups * p.waves * 64;
  return p;
}
static int64_t norm_back_lds(const NormSplit& p) {
  const int lanes = p.waves > 1 ? p.waves * 64 : 1 << p.lt;
  const int64_t vectors = (int64_t)2 * p.pieces * kPiece * 4 * 64 * p.waves;
  const int64_t handed = (int64_t)2 * p.pieces * kPiece * 4 * (p.slots / 2) * lanes;
  return std::max(vectors, handed);
}

// workgroups of the gradient: one per CU (its registers allow one), so that their column
// sums stay small beside the rows
static int norm_groups(int T, const NormSplit& p) { return (int)std::min<int64_t>(ceil_div(T, p.slots), 256); }

static int check_norm(const char* fn, const moe_block_norm_args* a) {
  MOE_CHECK_ARG(a != nullptr, MOE_ERR_INVALID_ARG, "%s: args is NULL", fn);
  MOE_CHECK_ARG(a->dtype >= MOE_BF16 && a->dtype <= MOE_FP32, MOE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, a->dtype);
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0, MOE_ERR_INVALID_ARG, "%s: bad sizes T=%d d=%d", fn, a->T, a->d);
  MOE_CHECK_ARG(a->d <= kNormMaxD && a->T <= (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: unsupported T=%d d=%d (T <= 2^24, d <= %d)", fn, a->T, a->d, kNormMaxD);
  MOE_CHECK_ARG((int64_t)a->T * a->d <= kMaxRowElements, MOE_ERR_UNSUPPORTED_SHAPE, "%s: unsupported T*d=%lld (<= 2^34)",
                fn, (long long)a->T * a->d);
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
  v.inv_d = 1.f / a->d;
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
  return (int64_t)std::min(T, 256) * 2 * d * 4;
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
  MOE_CHECK_ARG(!vectors || a->gate || a->gate_kind != MOE_GATE_CHANNEL, MOE_ERR_INVALID_ARG, "%s: gate is NULL", fn);
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
  v.dv_out = g->dnorm_out;
  v.dv_in = g->dnorm_in;
  v.dgate_vec = dgate_vec;
  hipStream_t s = (hipStream_t)stream;
  const NormSplit p = norm_back_split(a->T, a->d, a->dtype);
  const int groups = norm_groups(a->T, p);
  timing_begin(K_BLOCK_NORM_BWD, s);
  with_dtype(a->dtype, [&](auto e) {
    using S = decltype(e);
    if (a->T > 0) {
      auto launch = [&](auto kernel) {
        const int64_t lds = norm_back_lds(p);
        if (lds > 65536)  // (rows of over 8192 elements)
          (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(p.threads), (unsigned)lds, s, v, p);
      };
      auto go = [&](auto pieces, auto sub) {
        constexpr int R = decltype(pieces)::value;
        constexpr bool kSub = decltype(sub)::value;
        if (a->gate_kind == MOE_GATE_FULL)
          launch(k_block_norm_backward<S, R, kSub, true>);
        else
          launch(k_block_norm_backward<S, R, kSub, false>);
      };
      using std::integral_constant;
      if (p.lt < 6)
        go(integral_constant<int, 1>{}, std::true_type{});
      else if (p.pieces == 1)
        go(integral_constant<int, 1>{}, std::false_type{});
      else if (p.pieces == 2)
        go(integral_constant<int, 2>{}, std::false_type{});
      else if (p.pieces == 3)
        go(integral_constant<int, 3>{}, std::false_type{});
      else
        go(integral_constant<int, 4>{}, std::false_type{});
    }
    if (vectors && groups != 1)
      hipLaunchKernelGGL(k_norm_vectors<S>, dim3((unsigned)ceil_div(a->d, 32), 2), dim3(1024), 0, s, v.part, groups, v);
  });
  timing_end(K_BLOCK_NORM_BWD, s);
  return check_launch(fn);
}

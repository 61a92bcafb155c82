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
  float* part;  // [workgroup][3][d]: sums for v_out, v_in and the channel gate; or null
};

// sum of v over the workgroup, in every thread
__device__ __forceinline__ float block_sum(float v, float* lds) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += lds[w];
  return s;
}

template <typename S>
__device__ __forceinline__ const S* row_ptr(const void* p, int64_t t, int64_t stride) {
  return static_cast<const S*>(p) + t * stride;
}
template <typename S>
__device__ __forceinline__ S* row_ptr(void* p, int64_t t, int64_t stride) {
  return static_cast<S*>(p) + t * stride;
}

template <typename S, int R>
__global__ __launch_bounds__(kNormMaxThreads) void k_block_norm(NormDev a) {
  __shared__ float lds[kNormMaxThreads / 64];
  const int64_t t = blockIdx.x;
  float h[R][kPiece], z[R][kPiece];
  float ss = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
    if (n <= 0) continue;
    load_piece(row_ptr<S>(a.x, t, a.x_stride) + c, n, h[r]);
    if (a.y) load_piece(row_ptr<S>(a.y, t, a.y_stride) + c, n, z[r]);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      h[r][i] *= a.scale;
      if (a.y) ss = fmaf(z[r][i], z[r][i], ss);
    }
  }
  const float ry = a.v_out ? rsqrtf(block_sum(ss, lds) / a.d + a.eps) : 1.f;
  const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(*row_ptr<S>(a.gate, t, a.gate_stride)) : 1.f;
  float hh = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
    if (n <= 0) continue;
    if (a.y) {
      float v[kPiece], g[kPiece];
      if (a.v_out) load_piece(static_cast<const S*>(a.v_out) + c, n, v);
      if (a.gate_kind == MOE_GATE_CHANNEL) load_piece(static_cast<const S*>(a.gate) + c, n, g);
      if (a.gate_kind == MOE_GATE_FULL) load_piece(row_ptr<S>(a.gate, t, a.gate_stride) + c, n, g);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const float zi = a.v_out ? z[r][i] * ry * v[i] : z[r][i];
        const float gi = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL ? g[i] : gt;
        h[r][i] = fmaf(gi, zi, h[r][i]);
      }
    }
    if (a.h) store_piece(row_ptr<S>(a.h, t, a.h_stride) + c, n, h[r]);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) hh = fmaf(h[r][i], h[r][i], hh);
  }
  if (!a.v_in) return;
  const float rh = rsqrtf(block_sum(hh, lds) / a.d + a.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
    if (n <= 0) continue;
    float v[kPiece];
    load_piece(static_cast<const S*>(a.v_in) + c, n, v);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] *= h[r][i] * rh;
    store_piece(row_ptr<S>(a.n, t, a.n_stride) + c, n, v);
  }
}

template <typename S, int R>
__global__ __launch_bounds__(kNormMaxThreads) void k_block_norm_backward(NormDev a) {
  __shared__ float lds[kNormMaxThreads / 64];
  float sum_out[R][kPiece], sum_in[R][kPiece], sum_gate[R][kPiece];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sum_out[r][i] = sum_in[r][i] = sum_gate[r][i] = 0.f;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float h[R][kPiece], y[R][kPiece], D[R][kPiece], u[R][kPiece], v[R][kPiece], g[R][kPiece];
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(*row_ptr<S>(a.gate, t, a.gate_stride)) : 1.f;
    float ss = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        h[r][i] = y[r][i] = D[r][i] = u[r][i] = 0.f;
        v[r][i] = 1.f;
        g[r][i] = gt;
      }
      if (n <= 0) continue;
      load_piece(row_ptr<S>(a.x, t, a.x_stride) + c, n, h[r]);
      if (a.y) load_piece(row_ptr<S>(a.y, t, a.y_stride) + c, n, y[r]);
      if (a.dh) load_piece(row_ptr<S>(a.dh, t, a.dh_stride) + c, n, D[r]);
      if (a.dn) load_piece(row_ptr<S>(a.dn, t, a.dn_stride) + c, n, u[r]);
      if (a.v_out) load_piece(static_cast<const S*>(a.v_out) + c, n, v[r]);
      if (a.gate_kind == MOE_GATE_CHANNEL) load_piece(static_cast<const S*>(a.gate) + c, n, g[r]);
      if (a.gate_kind == MOE_GATE_FULL) load_piece(row_ptr<S>(a.gate, t, a.gate_stride) + c, n, g[r]);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) ss = fmaf(y[r][i], y[r][i], ss);
    }
    const float ry = a.v_out ? rsqrtf(block_sum(ss, lds) / a.d + a.eps) : 1.f;
    if (a.dn) {
      float hh = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const float z = y[r][i] * ry * v[r][i];
          h[r][i] = fmaf(g[r][i], z, a.scale * h[r][i]);
          hh = fmaf(h[r][i], h[r][i], hh);
        }
      const float rh = rsqrtf(block_sum(hh, lds) / a.d + a.eps);
      float m = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
        if (n <= 0) continue;
        float w[kPiece];
        load_piece(static_cast<const S*>(a.v_in) + c, n, w);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          h[r][i] *= rh;
          sum_in[r][i] = fmaf(u[r][i], h[r][i], sum_in[r][i]);
          u[r][i] *= w[i];
          m = fmaf(u[r][i], h[r][i], m);
        }
      }
      m = block_sum(m, lds) / a.d;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) D[r][i] = fmaf(rh, u[r][i] - h[r][i] * m, D[r][i]);
    }
    float m = 0.f, dg = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
      if (n <= 0) continue;
      float o[kPiece];
      if (a.dx) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) o[i] = a.scale * D[r][i];
        store_piece(row_ptr<S>(a.dx, t, a.dx_stride) + c, n, o);
      }
      if (!a.y) continue;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        y[r][i] *= ry;
        o[i] = D[r][i] * y[r][i] * v[r][i];
        dg += o[i];
        if (a.gate_kind == MOE_GATE_CHANNEL) sum_gate[r][i] += o[i];
        D[r][i] *= g[r][i];
        sum_out[r][i] = fmaf(D[r][i], y[r][i], sum_out[r][i]);
        D[r][i] *= v[r][i];
        m = fmaf(D[r][i], y[r][i], m);
      }
      if (a.gate_kind == MOE_GATE_FULL && a.dgate) store_piece(row_ptr<S>(a.dgate, t, a.dgate_stride) + c, n, o);
    }
    if (!a.y) continue;
    if (a.gate_kind == MOE_GATE_TOKEN && a.dgate) {
      dg = block_sum(dg, lds);
      if (threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = dg;
    }
    if (!a.dy) continue;
    m = a.v_out ? block_sum(m, lds) / a.d : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
      if (n <= 0) continue;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) D[r][i] = ry * (D[r][i] - y[r][i] * m);
      store_piece(row_ptr<S>(a.dy, t, a.dy_stride) + c, n, D[r]);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * kPiece, n = a.d - c;
    if (n <= 0) continue;
    float* p = a.part + (int64_t)blockIdx.x * 3 * a.d + c;
    store_piece(p, n, sum_out[r]);
    store_piece(p + a.d, n, sum_in[r]);
    store_piece(p + 2 * (int64_t)a.d, n, sum_gate[r]);
  }
}

// column sums of the workgroups' partial sums; blockIdx.y picks the vector
__global__ __launch_bounds__(256) void k_norm_vectors(const float* part, int groups, int d, float* dv_out,
                                                      float* dv_in, float* dgate) {
  float* out = blockIdx.y == 0 ? dv_out : blockIdx.y == 1 ? dv_in : dgate;
  if (!out) return;
  __shared__ float lds[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < d)
    for (int g = wave; g < groups; g += 4) s += part[((int64_t)g * 3 + blockIdx.y) * d + c];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) out[c] = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
}

// workgroups of the gradient: enough for every CU, few enough that their partial sums
// stay small beside the rows
static int norm_groups(int T) { return (int)std::min<int64_t>(T, 1024); }

struct NormShape {
  int threads, pieces;  // pieces of 8 elements per thread: 1 or 2
};
static NormShape norm_shape(int d) {
  const int lanes = (int)ceil_div(d, kPiece);
  if (lanes <= kNormMaxThreads) return {(int)ceil_div(lanes, 64) * 64, 1};
  return {kNormMaxThreads, 2};
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
  const NormShape sh = norm_shape(a->d);
  timing_begin(K_BLOCK_NORM, s);
  with_dtype(a->dtype, [&](auto e) {
    using S = decltype(e);
    if (sh.pieces == 1)
      hipLaunchKernelGGL((k_block_norm<S, 1>), dim3((unsigned)a->T), dim3(sh.threads), 0, s, v);
    else
      hipLaunchKernelGGL((k_block_norm<S, 2>), dim3((unsigned)a->T), dim3(sh.threads), 0, s, v);
  });
  timing_end(K_BLOCK_NORM, s);
  return check_launch(fn);
}

extern "C" int64_t moe_block_norm_backward_workspace_bytes(int T, int d) {
  if (T < 0 || d <= 0) return -1;
  return (int64_t)norm_groups(T) * 3 * d * 4;
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
  const NormShape sh = norm_shape(a->d);
  const int groups = norm_groups(a->T);
  timing_begin(K_BLOCK_NORM_BWD, s);
  if (a->T > 0)
    with_dtype(a->dtype, [&](auto e) {
      using S = decltype(e);
      if (sh.pieces == 1)
        hipLaunchKernelGGL((k_block_norm_backward<S, 1>), dim3(groups), dim3(sh.threads), 0, s, v);
      else
        hipLaunchKernelGGL((k_block_norm_backward<S, 2>), dim3(groups), dim3(sh.threads), 0, s, v);
    });
  if (vectors)
    hipLaunchKernelGGL(k_norm_vectors, dim3((unsigned)ceil_div(a->d, 64), 3), dim3(256), 0, s, v.part, groups, a->d,
                       g->dnorm_out, g->dnorm_in, dgate_vec);
  timing_end(K_BLOCK_NORM_BWD, s);
  return check_launch(fn);
}

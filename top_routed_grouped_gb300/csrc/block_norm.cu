// The join between two blocks: norm after a block, gate, scaled residual sum
// and norm before the next block, forward and backward (contracts with
// moe_block_norm in moe.h).
//
// A row belongs to a group of threads, 4 to 32 lanes of a warp for short
// rows and a whole CTA for others, and stays in registers between its loads
// and its stores: every input is read once.  A row's statistics are summed in
// an order set by H and the load width alone, so its outputs do not depend on
// the other rows.
//
// Backward: with v = r_out, x = v rstd the normed row and g = dh w,
//   dr = dr_out + rstd g - v c,   c = rstd^3 mean(g v)
// (the derivative of v -> v rsqrt(mean v^2 + eps)), and the same once more for
// y with u = scale gate dr in place of dh.  The row's first round of sums
// (v^2, g v, y^2) gives dr, the second (u w y) gives dy.  The gradients of
// the weights are sums over rows: each group keeps those of its own rows in
// registers, writes them once, and a second kernel adds the groups in order.
#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"

namespace moe {

constexpr int BN_MAX_THREADS = 512;

// ---- loads and stores of VEC neighbouring elements as floats ----
template <typename T, int VEC>
__device__ inline void bn_load(const T *p, float (&o)[VEC]) {
  if constexpr (VEC == 1) {
    o[0] = Elem<T>::load(p);
  } else {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int b = 0; b < VEC / N; ++b) {
      float v[N];
      Vec16<T>::load(p + b * N, v);
#pragma unroll
      for (int i = 0; i < N; ++i) o[b * N + i] = v[i];
    }
  }
}
template <typename T, int VEC>
__device__ inline void bn_store(T *p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = Elem<T>::from_f32(v[0]);
  } else {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int b = 0; b < VEC / N; ++b) {
      float o[N];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = v[b * N + i];
      Vec16<T>::store(p + b * N, o);
    }
  }
}
// Weights and channel gates: float or the rows' type.
template <typename T, int VEC>
__device__ inline void bn_load_w(const void *p, int i, bool f32, float add, float (&o)[VEC]) {
  if (f32) {
    if constexpr (VEC == 1) o[0] = ((const float *)p)[i];
    else bn_load<float, VEC>((const float *)p + i, o);
  } else {
    bn_load<T, VEC>((const T *)p + i, o);
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) o[k] += add;
}

// Sums of N values over the threads of a row, in a fixed order; all get them.
template <int N>
__device__ inline void bn_row_sum(float (&v)[N], int group, float *buf) {
  const int top = group < 32 ? group : 32;
  for (int d = top >> 1; d; d >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(FULL_MASK, v[n], d);
  if (group > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = group >> 5;
    __syncthreads();  // the buffer's last readers are done
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[n * 32 + warp] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0.f;
      for (int w = 0; w < warps; ++w) s += buf[n * 32 + w];
      v[n] = s;
    }
  }
}

template <typename TE, int VEC>
__device__ inline void bn_gate(const NormArgs &a, int64_t t, int i, float (&g)[VEC]) {
  if (a.gate_kind == MOE_GATE_ELEMENT) {
    bn_load<TE, VEC>((const TE *)a.gate + t * a.ld_gate + i, g);
  } else if (a.gate_kind == MOE_GATE_CHANNEL) {
    bn_load_w<TE, VEC>(a.gate, i, a.wf32, 0.f, g);
  } else {
    const float s = a.gate_kind == MOE_GATE_TOKEN ? ((const float *)a.gate)[t] : 1.f;
#pragma unroll
    for (int k = 0; k < VEC; ++k) g[k] = s;
  }
}

template <typename TE, typename TR, int VEC, int CH>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_kernel(const NormArgs a, int group) {
  __shared__ float buf[32];
  griddep_launch();
  griddep_wait();
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  for (int64_t t0 = (int64_t)blockIdx.x * per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * per_cta) {
    const bool row = t0 + sub < a.T;
    const int64_t t = row ? t0 + sub : a.T - 1;
    float v[CH][VEC], y[CH][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * group + lane) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[c][k] = y[c][k] = 0.f;
      if (i < a.H) {
        bn_load<TR, VEC>((const TR *)a.r + t * a.ld_r + i, v[c]);
        if (a.y) bn_load<TE, VEC>((const TE *)a.y + t * a.ld_y + i, y[c]);
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[0] = fmaf(y[c][k], y[c][k], s[0]);
    }
    if (a.y) {
      float rstd = 1.f;
      if (a.w_post) {
        bn_row_sum(s, group, buf);
        rstd = rsqrtf(fmaf(s[0], inv_h, a.eps));
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i < a.H) {
          float g[VEC];
          bn_gate<TE, VEC>(a, t, i, g);
          if (a.w_post) {
            float w[VEC];
            bn_load_w<TE, VEC>(a.w_post, i, a.wf32, a.offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) y[c][k] *= rstd * w[k];
          }
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[c][k] = fmaf(a.scale * g[k], y[c][k], v[c][k]);
          if (row) bn_store<TR, VEC>((TR *)a.r_out + t * a.ld_r_out + i, v[c]);
        }
      }
    }
    if (a.w_pre) {
      s[0] = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[0] = fmaf(v[c][k], v[c][k], s[0]);
      bn_row_sum(s, group, buf);
      const float rstd = rsqrtf(fmaf(s[0], inv_h, a.eps));
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i < a.H && row) {
          float w[VEC];
          bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) w[k] *= v[c][k] * rstd;
          bn_store<TE, VEC>((TE *)a.h + t * a.ld_h + i, w);
        }
      }
    }
  }
}

// part: [3][groups][H] sums over a group's rows of what dw_pre, dw_post and a
// channel gate's gradient are made of (only those that the call asks for).
template <typename TE, typename TR, int VEC, int CH>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_bwd_kernel(const NormArgs a, int group, float *part) {
  __shared__ float buf[3 * 32];
  griddep_launch();
  griddep_wait();
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  float dwa[CH][VEC], dwb[CH][VEC], dga[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dwa[c][k] = dwb[c][k] = dga[c][k] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * per_cta) {
    const bool row = t0 + sub < a.T;
    const int64_t t = row ? t0 + sub : a.T - 1;
    float v[CH][VEC], d[CH][VEC], y[CH][VEC], e[CH][VEC];
    float s[3] = {0.f, 0.f, 0.f};  // v^2, dh w v, y^2
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * group + lane) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[c][k] = d[c][k] = y[c][k] = e[c][k] = 0.f;
      if (i < a.H) {
        if (a.dr_out) bn_load<TR, VEC>((const TR *)a.dr_out + t * a.ld_dr_out + i, e[c]);
        if (a.w_pre) {
          bn_load<TR, VEC>((const TR *)a.r_out + t * a.ld_r_out + i, v[c]);
          bn_load<TE, VEC>((const TE *)a.dh + t * a.ld_dh + i, d[c]);
        }
        if (a.y) bn_load<TE, VEC>((const TE *)a.y + t * a.ld_y + i, y[c]);
      }
      if (a.w_pre && i < a.H) {
        float w[VEC];
        bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          s[0] = fmaf(v[c][k], v[c][k], s[0]);
          s[1] = fmaf(d[c][k] * w[k], v[c][k], s[1]);
        }
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[2] = fmaf(y[c][k], y[c][k], s[2]);
    }
    bn_row_sum(s, group, buf);
    if (a.w_pre) {
      const float rstd = rsqrtf(fmaf(s[0], inv_h, a.eps)), cr = s[1] * inv_h * rstd * rstd * rstd;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i < a.H) {
          float w[VEC];
          bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            if (row) dwa[c][k] = fmaf(d[c][k], v[c][k] * rstd, dwa[c][k]);
            e[c][k] += fmaf(d[c][k] * w[k], rstd, -v[c][k] * cr);
          }
          if (row) bn_store<TR, VEC>((TR *)a.dr + t * a.ld_dr + i, e[c]);
        }
      }
    }
    if (a.y) {
      const float rstd = a.w_post ? rsqrtf(fmaf(s[2], inv_h, a.eps)) : 1.f;
      float q[2] = {0.f, 0.f};  // u w y, scale dr w y
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i < a.H) {
          float g[VEC], w[VEC], dg[VEC];
          bn_gate<TE, VEC>(a, t, i, g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) w[k] = 1.f;
          if (a.w_post) bn_load_w<TE, VEC>(a.w_post, i, a.wf32, a.offset, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float se = a.scale * e[c][k], x = y[c][k] * rstd, u = se * g[k];
            dg[k] = se * w[k] * x;
            q[0] = fmaf(u * w[k], y[c][k], q[0]);
            q[1] += dg[k];
            if (row) dwb[c][k] = fmaf(u, x, dwb[c][k]);
            if (row) dga[c][k] += dg[k];
            d[c][k] = u * w[k] * rstd;
          }
          if (a.gate_kind == MOE_GATE_ELEMENT && row) bn_store<TE, VEC>((TE *)a.dgate + t * a.ld_dgate + i, dg);
        }
      }
      float cy = 0.f;
      if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) {
        bn_row_sum(q, group, buf);
        if (a.w_post) cy = q[0] * inv_h * rstd * rstd * rstd;
        if (a.gate_kind == MOE_GATE_TOKEN && lane == 0 && row) ((float *)a.dgate)[t] = q[1];
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i < a.H && row) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) d[c][k] = fmaf(-y[c][k], cy, d[c][k]);
          bn_store<TE, VEC>((TE *)a.dy + t * a.ld_dy + i, d[c]);
        }
      }
    }
  }
  const int64_t groups = (int64_t)gridDim.x * per_cta;
  float *p = part + ((int64_t)blockIdx.x * per_cta + sub) * a.H;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int i = (c * group + lane) * VEC + k;
      if (i < a.H) {
        if (a.dw_pre) p[i] = dwa[c][k];
        if (a.dw_post) p[groups * a.H + i] = dwb[c][k];
        if (a.gate_kind == MOE_GATE_CHANNEL) p[2 * groups * a.H + i] = dga[c][k];
      }
    }
}

// out[i] = sum over the groups of part[.][i], in a fixed order: 32 threads of
// a column take every 32nd group, then a tree.
__global__ void __launch_bounds__(1024) block_norm_join_kernel(const float *part, int64_t groups, int H, float *o0,
                                                               float *o1, float *o2) {
  __shared__ float buf[32][33];
  griddep_launch();
  griddep_wait();
  float *out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int i = blockIdx.x * 32 + threadIdx.x;
  const float *p = part + (int64_t)blockIdx.y * groups * H;
  float s = 0.f;
  if (i < H)
    for (int64_t g = threadIdx.y; g < groups; g += 32) s += p[g * H + i];
  buf[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  float v = buf[threadIdx.x][threadIdx.y];  // column threadIdx.y, group slot threadIdx.x
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  if (threadIdx.x == 0 && (int)blockIdx.x * 32 + (int)threadIdx.y < H) out[blockIdx.x * 32 + threadIdx.y] = v;
}

// ---------------------------------------------------------------- host
// Threads of a row (a power of two up to 32, or a multiple of 32), chunks of
// the load width in each, threads of a CTA.
struct BnShape {
  int vec, ch, group, threads;
};

static bool bn_wide(const NormArgs &a, int vec) {
  auto row = [&](const void *p, int64_t ld, int es) { return !p || (((uintptr_t)p & 15) == 0 && ld * es % 16 == 0); };
  const int e = a.f32 ? 4 : 2, r = a.rf32 ? 4 : 2;
  bool ok = a.H % vec == 0 && row(a.r, a.ld_r, r) && row(a.y, a.ld_y, e) && row(a.r_out, a.ld_r_out, r) &&
            row(a.h, a.ld_h, e) && row(a.dr_out, a.ld_dr_out, r) && row(a.dh, a.ld_dh, e) && row(a.dr, a.ld_dr, r) &&
            row(a.dy, a.ld_dy, e) && row(a.w_post, 0, 1) && row(a.w_pre, 0, 1);
  if (a.gate_kind == MOE_GATE_CHANNEL) ok = ok && row(a.gate, 0, 1);
  if (a.gate_kind == MOE_GATE_ELEMENT) ok = ok && row(a.gate, a.ld_gate, e) && row(a.dgate, a.ld_dgate, e);
  return ok;
}

static BnShape bn_shape(const NormArgs &a) {
  BnShape s;
  s.vec = a.f32 ? 4 : 8;
  if (!bn_wide(a, s.vec)) s.vec = 1;
  const int n = (int)ceil_div(a.H, s.vec);
  const int wide[3] = {1, 2, s.vec == 4 ? 8 : 4}, scalar[3] = {2, 8, 32};
  const int *opt = s.vec == 1 ? scalar : wide;
  int i = 0;
  while (i < 2 && ceil_div(n, opt[i]) > 256) ++i;
  s.ch = opt[i];
  const int need = (int)ceil_div(n, s.ch);
  if (need <= 32) {
    s.group = 4;
    while (s.group < need) s.group *= 2;
    s.threads = 256;
  } else {
    s.group = (int)round_up(need, 32);
    s.threads = s.group;
  }
  return s;
}

template <typename TE, typename TR, int VEC, int CH>
static cudaError_t bn_launch(const NormArgs &a, const BnShape &s, int grid, float *part, cudaStream_t stream) {
  if (part) return launch_pdl(block_norm_bwd_kernel<TE, TR, VEC, CH>, dim3(grid), dim3(s.threads), 0, stream, a, s.group, part);
  return launch_pdl(block_norm_kernel<TE, TR, VEC, CH>, dim3(grid), dim3(s.threads), 0, stream, a, s.group);
}

template <typename TE, typename TR>
static cudaError_t bn_dispatch(const NormArgs &a, const BnShape &s, int grid, float *part, cudaStream_t stream) {
  constexpr int W = Vec16<TE>::N;
  if (s.vec == 1) {
    if (s.ch == 2) return bn_launch<TE, TR, 1, 2>(a, s, grid, part, stream);
    if (s.ch == 8) return bn_launch<TE, TR, 1, 8>(a, s, grid, part, stream);
    return bn_launch<TE, TR, 1, 32>(a, s, grid, part, stream);
  }
  if (s.ch == 1) return bn_launch<TE, TR, W, 1>(a, s, grid, part, stream);
  if (s.ch == 2) return bn_launch<TE, TR, W, 2>(a, s, grid, part, stream);
  return bn_launch<TE, TR, W, 32 / W>(a, s, grid, part, stream);
}

static cudaError_t bn_any(const NormArgs &a, const BnShape &s, int grid, float *part, cudaStream_t stream) {
  if (a.f32) return bn_dispatch<float, float>(a, s, grid, part, stream);
  if (a.rf32) return bn_dispatch<__nv_bfloat16, float>(a, s, grid, part, stream);
  return bn_dispatch<__nv_bfloat16, __nv_bfloat16>(a, s, grid, part, stream);
}

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const BnShape s = bn_shape(a);
  const int64_t ctas = ceil_div(a.T, s.threads / s.group);
  return bn_any(a, s, (int)(ctas < (1 << 30) ? ctas : 1 << 30), nullptr, stream);
}

// CTAs of the backward: enough to fill the device, no more than the rows need.
static int bn_bwd_grid(const NormArgs &a, const BnShape &s) {
  const int64_t fill = (int64_t)device_sms() * (1024 / s.threads > 0 ? 1024 / s.threads : 1);
  const int64_t ctas = ceil_div(a.T, s.threads / s.group);
  return (int)(ctas < fill ? ctas : fill);
}

size_t block_norm_scratch_bytes(const NormArgs &a) {
  if (a.T == 0) return 0;
  const BnShape s = bn_shape(a);
  return (size_t)3 * bn_bwd_grid(a, s) * (s.threads / s.group) * a.H * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const NormArgs &a, void *scratch, cudaStream_t stream) {
  float *dg = a.gate_kind == MOE_GATE_CHANNEL ? (float *)a.dgate : nullptr;
  if (a.T == 0) {
    cudaError_t e = cudaSuccess;
    for (float *p : {a.dw_pre, a.dw_post, dg})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)a.H * 4, stream);
    return e;
  }
  const BnShape s = bn_shape(a);
  const int grid = bn_bwd_grid(a, s);
  cudaError_t e = bn_any(a, s, grid, (float *)scratch, stream);
  if (e != cudaSuccess || (!a.dw_pre && !a.dw_post && !dg)) return e;
  return launch_pdl(block_norm_join_kernel, dim3((unsigned)ceil_div(a.H, 32), 3), dim3(32, 32), 0, stream,
                    (const float *)scratch, (int64_t)grid * (s.threads / s.group), a.H, a.dw_pre, a.dw_post, dg);
}

}  // namespace moe

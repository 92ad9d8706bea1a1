// The join between two blocks: norm after a block, gate, scaled residual sum
// and norm before the next block, forward and backward (contracts with
// moe_block_norm in moe.h).
//
// A row belongs to a group of threads, 4 to 32 lanes of a warp for short
// rows and a whole CTA for others, and stays in registers between its loads
// and its stores: every input is read once.  CTAs walk over the rows; the
// inputs of the next few blocks of rows are on their way to shared memory by
// bulk copies meanwhile.  A row that starts between 16-byte boundaries is
// copied with the bytes around it, so odd widths move as fast.  A group takes
// two rows at a time where they are short, so that the rounds of a sum over a row, which are
// latency, are shared.  Rows too long for two such stages are loaded straight
// from memory.  A row's statistics
// are summed in an order set by H and the load width alone, so its outputs do
// not depend on the other rows.
//
// Backward: with v = r_out, x = v rstd the normed row and g = dh w,
//   dr = dr_out + rstd g - v c,   c = rstd^3 mean(g v)
// (the derivative of v -> v rsqrt(mean v^2 + eps)), and the same once more for
// y with u = scale gate dr in place of dh.  The row's first round of sums
// (v^2, g v, y^2) gives dr, the second (u w y) gives dy.  The gradients of
// the weights are sums over rows: each group keeps those of its own rows in
// registers, writes them once, and a second kernel adds the groups in order.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int BN_MAX_THREADS = 512, BN_MAX_STAGES = 6, BN_MAX_INPUTS = 5;

// The row inputs of a launch and where their blocks of rows stand in a stage.
struct BnStages {
  int n, stages, bytes;  // inputs, stages, bytes of a stage
  int rows;              // of a block
  int runs;              // runs of bytes that it is: 1 (rows behind one another), or its rows
  int off[BN_MAX_INPUTS], es[BN_MAX_INPUTS], pitch[BN_MAX_INPUTS];  // pitch: bytes from run to run in a stage
  int64_t ld[BN_MAX_INPUTS];
  const void *base[BN_MAX_INPUTS];
};

struct BnBars {
  uint64_t full[BN_MAX_STAGES];
  int abort_flag;
};

// The bytes that run `q` of input k of block `t0` copies: the 16-byte pieces
// that its rows touch, none outside the buffer; and its rows' own bytes.
struct BnPiece {
  uintptr_t from, to, lo, hi;  // [from, to) is copied; the rows are [lo, hi)
};
__device__ inline BnPiece bn_piece(const BnStages &st, int k, int q, int64_t t0, int T, int H) {
  const int64_t first_row = t0 + q, rows = st.runs > 1 ? 1 : min((int64_t)st.rows, T - t0);
  BnPiece p = {0, 0, 0, 0};
  if (first_row >= T) return p;
  p.lo = (uintptr_t)st.base[k] + first_row * st.ld[k] * st.es[k];
  p.hi = p.lo + ((rows - 1) * st.ld[k] + H) * st.es[k];
  const uintptr_t first = ((uintptr_t)st.base[k] + 15) & ~(uintptr_t)15;
  const uintptr_t last = ((uintptr_t)st.base[k] + ((T - 1) * st.ld[k] + H) * st.es[k]) & ~(uintptr_t)15;
  p.from = max(p.lo & ~(uintptr_t)15, first);
  p.to = min((p.hi + 15) & ~(uintptr_t)15, last);
  if (p.to < p.from) p.from = p.to = p.hi;
  return p;
}
// Starts the copies of a block (one warp; at most 32 of them).
__device__ inline void bn_start(const BnStages &st, uint8_t *stage, uint64_t *bar, int64_t t0, int T, int H) {
  const int lane = threadIdx.x & 31, k = lane / st.runs, q = lane % st.runs;
  BnPiece p = {0, 0, 0, 0};
  if (k < st.n) p = bn_piece(st, k, q, t0, T, H);
  const uint32_t bytes = (uint32_t)(p.to - p.from);
  const uint32_t all = __reduce_add_sync(FULL_MASK, bytes);
  if (lane == 0) {
    if (all) umma::mbar_arrive_expect_tx(bar, all);
    else umma::mbar_arrive(bar);
  }
  __syncwarp();
  if (bytes)
    umma::bulk_load(stage + st.off[k] + q * st.pitch[k] + (p.from - (p.lo & ~(uintptr_t)15)), (const void *)p.from, bytes, bar);
}
// What the copies of the first and the last block may have missed (the whole
// CTA; the caller's barrier follows).
__device__ inline bool bn_mend(const BnStages &st, uint8_t *stage, int64_t t0, int T, int H) {
  if (t0 > 0 && t0 + st.rows < T) return false;
  bool missed = false;
  for (int k = 0; k < st.n; ++k)
    for (int q = 0; q < st.runs; ++q) {
      const BnPiece p = bn_piece(st, k, q, t0, T, H);
      if (p.from <= p.lo && p.to >= p.hi) continue;
      missed = true;
      uint8_t *dst = stage + st.off[k] + q * st.pitch[k] - (p.lo & ~(uintptr_t)15);
      for (uintptr_t b = p.lo + threadIdx.x; b < p.hi; b += blockDim.x)
        if (b < p.from || b >= p.to) dst[b] = *(const uint8_t *)b;
    }
  return missed;
}

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
// Consecutive calls alternate between two buffers: the barrier of one call
// tells that the buffer of the call before it has been read.
template <int N>
__device__ inline void bn_row_sum(float (&v)[N], int group, float (*buf)[16]) {
  const int top = group < 32 ? group : 32;
  for (int d = top >> 1; d; d >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(FULL_MASK, v[n], d);
  if (group > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = group >> 5;
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[n][warp] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = 0.f;
    for (int w = 0; w < warps; w += 4)  // (slots past the last warp hold zeros)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float4 f = *(const float4 *)&buf[n][w];
        v[n] += f.x;
        v[n] += f.y;
        v[n] += f.z;
        v[n] += f.w;
      }
  }
}

template <typename TE, int VEC>
__device__ inline void bn_gate(const NormArgs &a, int64_t t, int i, const void *elements, float (&g)[VEC]) {
  if (a.gate_kind == MOE_GATE_ELEMENT) {
    bn_load<TE, VEC>((const TE *)elements + i, g);
  } else if (a.gate_kind == MOE_GATE_CHANNEL) {
    bn_load_w<TE, VEC>(a.gate, i, a.wf32, 0.f, g);
  } else {
    const float s = a.gate_kind == MOE_GATE_TOKEN ? ((const float *)a.gate)[t] : 1.f;
#pragma unroll
    for (int k = 0; k < VEC; ++k) g[k] = s;
  }
}

// A CTA's walk over its blocks of rows, with stages (BULK) or without.
template <bool BULK, int R>
struct BnWalk {
  const BnStages &st;
  const int T, H, per_cta;
  const int64_t step;
  uint8_t *stages, *stage;
  BnBars &bars;
  int64_t t0;
  int slot = 0;
  uint32_t phase = 0;
  bool first = true;

  __device__ inline BnWalk(const BnStages &s, int T_, int H_, int per_cta_, uint8_t *stages_, BnBars &b)
      : st(s), T(T_), H(H_), per_cta(per_cta_), step((int64_t)gridDim.x * per_cta_ * R), stages(stages_), stage(stages_),
        bars(b), t0((int64_t)blockIdx.x * per_cta_ * R) {
    if (BULK) {
      if (threadIdx.x == 0) {
        for (int i = 0; i < st.stages; ++i) umma::mbar_init(&bars.full[i], 1);
        umma::fence_mbar_init();
        bars.abort_flag = 0;
      }
      __syncthreads();
    }
    griddep_launch();
    griddep_wait();
    if (BULK && threadIdx.x < 32)
      for (int i = 0; i < st.stages; ++i)
        if (t0 + i * step < T) bn_start(st, stages + i * st.bytes, &bars.full[i], t0 + i * step, T, H);
  }
  // Waits for the block's stage.
  __device__ inline bool arrive(int *status) {
    if (!BULK) return true;
    stage = stages + slot * st.bytes;
    if (!umma::mbar_wait(&bars.full[slot], phase, &bars.abort_flag, status)) return false;
    if (bn_mend(st, stage, t0, T, H)) __syncthreads();
    return true;
  }
  // Row t (the j-th of the block) of staged input k, or of `p` in memory.
  template <typename E>
  __device__ inline const E *row(int k, const void *p, int64_t ld, int64_t t, int j) const {
    if (!BULK) return (const E *)p + t * ld;
    if (st.runs > 1) {
      const uintptr_t at = (uintptr_t)p + t * ld * sizeof(E);
      return (const E *)(stage + st.off[k] + j * st.pitch[k] + (at & 15));
    }
    const uintptr_t at = (uintptr_t)p + t0 * ld * sizeof(E);
    return (const E *)(stage + st.off[k] + (at & 15)) + (t - t0) * ld;
  }
  // Behind a barrier of this block: the last block's stage has been read by
  // all, its copies for a later block start.
  __device__ inline void refill() {
    if (BULK && !first && threadIdx.x < 32) {
      const int old = slot ? slot - 1 : st.stages - 1;
      const int64_t later = t0 - step + st.stages * step;
      if (later < T) bn_start(st, stages + old * st.bytes, &bars.full[old], later, T, H);
    }
    first = false;
  }
  __device__ inline void next() {
    t0 += step;
    if (++slot == st.stages) slot = 0, phase ^= 1;
  }
};

// Threads of an SM that the kernels' registers allow.
constexpr int bn_resident(bool backward, int vec, int ch) { return !backward && vec * ch <= 8 ? 1024 : 512; }

template <typename TE, typename TR, int VEC, int CH, int R, bool BULK>
__global__ void __launch_bounds__(BN_MAX_THREADS, bn_resident(false, VEC, CH) / BN_MAX_THREADS)
block_norm_kernel(const NormArgs a, int group, const BnStages st, int *status) {
  extern __shared__ __align__(128) uint8_t bn_smem[];
  __shared__ BnBars bars;
  __shared__ __align__(16) float buf[2][R][16];
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  if (threadIdx.x < 2 * R * 16) buf[0][0][threadIdx.x] = 0.f;
  if (!BULK) __syncthreads();
  BnWalk<BULK, R> walk(st, a.T, a.H, per_cta, bn_smem, bars);
  int round = 0;
  for (; walk.t0 < a.T; walk.next()) {
    if (!walk.arrive(status)) return;
    int64_t t[R];
    bool row[R];
    float s[R], rstd[R], v[R][CH][VEC];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      t[j] = walk.t0 + j * per_cta + sub;
      row[j] = t[j] < a.T;
      if (!row[j]) t[j] = walk.t0 + sub < a.T ? walk.t0 + sub : walk.t0;  // (some row of the block)
      s[j] = 0.f;
      rstd[j] = 1.f;
    }
    auto at = [&](int j) { return row[j] ? j * per_cta + sub : (int)(t[j] - walk.t0); };
    if (a.w_post) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const TE *y_in = walk.template row<TE>(1, a.y, a.ld_y, t[j], at(j));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = (c * group + lane) * VEC;
          float y[VEC];
          if (i < a.H) {
            bn_load<TE, VEC>(y_in + i, y);
#pragma unroll
            for (int k = 0; k < VEC; ++k) s[j] = fmaf(y[k], y[k], s[j]);
          }
        }
      }
      bn_row_sum(s, group, buf[round++ & 1]);
#pragma unroll
      for (int j = 0; j < R; ++j) rstd[j] = rsqrtf(fmaf(s[j], inv_h, a.eps));
    }
    if (BULK && (!a.w_post || group <= 32)) __syncthreads();
    walk.refill();
#pragma unroll
    for (int j = 0; j < R; ++j) {
      s[j] = 0.f;
      const TR *r_in = walk.template row<TR>(0, a.r, a.ld_r, t[j], at(j));
      const TE *y_in = a.y ? walk.template row<TE>(1, a.y, a.ld_y, t[j], at(j)) : nullptr;
      const void *g_in = a.gate_kind == MOE_GATE_ELEMENT ? walk.template row<TE>(2, a.gate, a.ld_gate, t[j], at(j)) : nullptr;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[j][c][k] = 0.f;
        if (i >= a.H) continue;
        bn_load<TR, VEC>(r_in + i, v[j][c]);
        if (a.y) {
          float y[VEC], g[VEC];
          bn_load<TE, VEC>(y_in + i, y);
          bn_gate<TE, VEC>(a, t[j], i, g_in, g);
          if (a.w_post) {
            float w[VEC];
            bn_load_w<TE, VEC>(a.w_post, i, a.wf32, a.offset, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) y[k] *= rstd[j] * w[k];
          }
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[j][c][k] = fmaf(a.scale * g[k], y[k], v[j][c][k]);
          if (row[j]) bn_store<TR, VEC>((TR *)a.r_out + t[j] * a.ld_r_out + i, v[j][c]);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[j] = fmaf(v[j][c][k], v[j][c][k], s[j]);
      }
    }
    if (a.w_pre) {
      bn_row_sum(s, group, buf[round++ & 1]);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
        if (i >= a.H) continue;
        float w[VEC];
        bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const float rs = rsqrtf(fmaf(s[j], inv_h, a.eps));
          float h[VEC];
#pragma unroll
          for (int k = 0; k < VEC; ++k) h[k] = w[k] * (v[j][c][k] * rs);
          if (row[j]) bn_store<TE, VEC>((TE *)a.h + t[j] * a.ld_h + i, h);
        }
      }
    }
  }
}

// part: [3][groups][H] sums over a group's rows of what dw_pre, dw_post and a
// channel gate's gradient are made of (only those that the call asks for).
template <typename TE, typename TR, int VEC, int CH, int R, bool BULK>
__global__ void __launch_bounds__(BN_MAX_THREADS)
block_norm_bwd_kernel(const NormArgs a, int group, const BnStages st, float *part, int *status) {
  extern __shared__ __align__(128) uint8_t bn_smem[];
  __shared__ BnBars bars;
  __shared__ __align__(16) float buf[2][3 * R][16];
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  for (int i = threadIdx.x; i < 2 * 3 * R * 16; i += blockDim.x) buf[0][0][i] = 0.f;
  if (!BULK) __syncthreads();
  float dwa[CH][VEC], dwb[CH][VEC], dga[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dwa[c][k] = dwb[c][k] = dga[c][k] = 0.f;
  // Inputs are staged in the order of their use.
  const int in_r = a.dr_out ? 1 : 0, in_d = in_r + 1, in_y = in_r + (a.w_pre ? 2 : 0), in_g = in_y + 1;
  BnWalk<BULK, R> walk(st, a.T, a.H, per_cta, bn_smem, bars);
  int round = 0;
  for (; walk.t0 < a.T; walk.next()) {
    if (!walk.arrive(status)) return;
    int64_t t[R];
    bool row[R];
    float s[3 * R], e[R][CH][VEC];  // s: v^2, dh w v, y^2 of each row
#pragma unroll
    for (int j = 0; j < R; ++j) {
      t[j] = walk.t0 + j * per_cta + sub;
      row[j] = t[j] < a.T;
      if (!row[j]) t[j] = walk.t0 + sub < a.T ? walk.t0 + sub : walk.t0;
      s[3 * j] = s[3 * j + 1] = s[3 * j + 2] = 0.f;
    }
    auto at = [&](int j) { return row[j] ? j * per_cta + sub : (int)(t[j] - walk.t0); };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * group + lane) * VEC;
      if (i >= a.H) continue;
      float w[VEC];
      if (a.w_pre) bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (a.w_pre) {
          float v[VEC], d[VEC];
          bn_load<TR, VEC>(walk.template row<TR>(in_r, a.r_out, a.ld_r_out, t[j], at(j)) + i, v);
          bn_load<TE, VEC>(walk.template row<TE>(in_d, a.dh, a.ld_dh, t[j], at(j)) + i, d);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            s[3 * j] = fmaf(v[k], v[k], s[3 * j]);
            s[3 * j + 1] = fmaf(d[k] * w[k], v[k], s[3 * j + 1]);
          }
        }
        if (a.w_post) {
          float y[VEC];
          bn_load<TE, VEC>(walk.template row<TE>(in_y, a.y, a.ld_y, t[j], at(j)) + i, y);
#pragma unroll
          for (int k = 0; k < VEC; ++k) s[3 * j + 2] = fmaf(y[k], y[k], s[3 * j + 2]);
        }
      }
    }
    bn_row_sum(s, group, buf[round++ & 1]);
    if (BULK && group <= 32) __syncthreads();
    walk.refill();
    float rv[R], cr[R], ry[R], q[2 * R];  // q: u w y, scale dr w y
#pragma unroll
    for (int j = 0; j < R; ++j) {
      rv[j] = rsqrtf(fmaf(s[3 * j], inv_h, a.eps));
      cr[j] = s[3 * j + 1] * inv_h * rv[j] * rv[j] * rv[j];
      ry[j] = a.w_post ? rsqrtf(fmaf(s[3 * j + 2], inv_h, a.eps)) : 1.f;
      q[2 * j] = q[2 * j + 1] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * group + lane) * VEC;
      if (i >= a.H) continue;
      float w[VEC], wp[VEC];
      if (a.w_pre) bn_load_w<TE, VEC>(a.w_pre, i, a.wf32, a.offset, w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) wp[k] = 1.f;
      if (a.w_post) bn_load_w<TE, VEC>(a.w_post, i, a.wf32, a.offset, wp);
#pragma unroll
      for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) e[j][c][k] = 0.f;
        if (a.dr_out) bn_load<TR, VEC>(walk.template row<TR>(0, a.dr_out, a.ld_dr_out, t[j], at(j)) + i, e[j][c]);
        if (a.w_pre) {
          float v[VEC], d[VEC];
          bn_load<TR, VEC>(walk.template row<TR>(in_r, a.r_out, a.ld_r_out, t[j], at(j)) + i, v);
          bn_load<TE, VEC>(walk.template row<TE>(in_d, a.dh, a.ld_dh, t[j], at(j)) + i, d);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            if (row[j]) dwa[c][k] = fmaf(d[k], v[k] * rv[j], dwa[c][k]);
            e[j][c][k] += fmaf(d[k] * w[k], rv[j], -v[k] * cr[j]);
          }
          if (row[j]) bn_store<TR, VEC>((TR *)a.dr + t[j] * a.ld_dr + i, e[j][c]);
        }
        if (a.y) {
          float y[VEC], g[VEC], dg[VEC];
          bn_load<TE, VEC>(walk.template row<TE>(in_y, a.y, a.ld_y, t[j], at(j)) + i, y);
          bn_gate<TE, VEC>(a, t[j], i, a.gate_kind == MOE_GATE_ELEMENT ? walk.template row<TE>(in_g, a.gate, a.ld_gate, t[j], at(j)) : nullptr, g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float se = a.scale * e[j][c][k], x = y[k] * ry[j], u = se * g[k];
            dg[k] = se * wp[k] * x;
            q[2 * j] = fmaf(u * wp[k], y[k], q[2 * j]);
            q[2 * j + 1] += dg[k];
            if (row[j]) {
              dwb[c][k] = fmaf(u, x, dwb[c][k]);
              dga[c][k] += dg[k];
            }
            e[j][c][k] = u * wp[k] * ry[j];  // dy but for its last term
          }
          if (a.gate_kind == MOE_GATE_ELEMENT && row[j]) bn_store<TE, VEC>((TE *)a.dgate + t[j] * a.ld_dgate + i, dg);
        }
      }
    }
    if (a.y) {
      if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) bn_row_sum(q, group, buf[round++ & 1]);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float cy = a.w_post ? q[2 * j] * inv_h * ry[j] * ry[j] * ry[j] : 0.f;
        if (a.gate_kind == MOE_GATE_TOKEN && lane == 0 && row[j]) ((float *)a.dgate)[t[j]] = q[2 * j + 1];
        const TE *y_in = walk.template row<TE>(in_y, a.y, a.ld_y, t[j], at(j));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = (c * group + lane) * VEC;
          if (i >= a.H || !row[j]) continue;
          if (a.w_post) {
            float y[VEC];
            bn_load<TE, VEC>(y_in + i, y);
#pragma unroll
            for (int k = 0; k < VEC; ++k) e[j][c][k] = fmaf(-y[k], cy, e[j][c][k]);
          }
          bn_store<TE, VEC>((TE *)a.dy + t[j] * a.ld_dy + i, e[j][c]);
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
  while (i < 2 && ceil_div(n, opt[i]) > BN_MAX_THREADS) ++i;
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

// The inputs that rows come from, in the order in which the kernels name them.
static BnStages bn_inputs(const NormArgs &a, bool backward) {
  BnStages st = {};
  const int e = a.f32 ? 4 : 2, r = a.rf32 ? 4 : 2;
  auto add = [&](const void *p, int64_t ld, int es) {
    if (!p) return;
    st.base[st.n] = p;
    st.ld[st.n] = ld;
    st.es[st.n++] = es;
  };
  const void *gate = a.gate_kind == MOE_GATE_ELEMENT ? a.gate : nullptr;
  if (backward) {
    add(a.dr_out, a.ld_dr_out, r);
    add(a.r_out, a.ld_r_out, r);
    add(a.dh, a.ld_dh, e);
    add(a.y, a.ld_y, e);
    add(gate, a.ld_gate, e);
  } else {
    add(a.r, a.ld_r, r);
    add(a.y, a.ld_y, e);
    add(gate, a.ld_gate, e);
  }
  return st;
}

constexpr int BN_SMEM = 220 * 1024;  // of an SM, for the stages of its CTAs

// Fills in the stages for `ctas` CTAs on an SM that take R rows a group; false
// where two stages do not fit, or short rows are not behind one another.
static bool bn_stages(const NormArgs &a, const BnShape &s, int ctas, int R, BnStages &st) {
  const int per_cta = s.threads / s.group;
  st.rows = per_cta * R;
  st.runs = 1;
  st.bytes = 0;
  for (int k = 0; k < st.n; ++k)
    if (st.rows > 1 && st.ld[k] != a.H) st.runs = st.rows;
  if (st.runs > 1 && (per_cta > 1 || st.runs * st.n > 32)) return false;
  for (int k = 0; k < st.n; ++k) {
    st.off[k] = st.bytes;
    st.pitch[k] = (int)round_up((int64_t)(st.runs > 1 ? 1 : st.rows) * a.H * st.es[k], 16) + 16;
    st.bytes += st.runs * st.pitch[k];
  }
  st.bytes = (int)round_up(st.bytes, 128);
  st.stages = std::min(BN_MAX_STAGES, BN_SMEM / ctas / st.bytes);
  return st.stages >= 2;
}

struct BnLaunch {
  const NormArgs &a;
  bool backward;
  float *part;
  int *status;
  cudaStream_t stream;
  int *groups;  // out: groups that leave partial sums
  bool dry;     // only `groups` is wanted
};

template <typename TE, typename TR, int VEC, int CH, int R, bool BULK>
static cudaError_t bn_go(const BnLaunch &l, const BnShape &s, int ctas, const BnStages &st) {
  const NormArgs &a = l.a;
  const int per_cta = s.threads / s.group;
  const int grid = (int)std::min<int64_t>(ceil_div(a.T, per_cta * R), (int64_t)device_sms() * ctas);
  if (l.groups) *l.groups = grid * per_cta;
  if (l.dry) return cudaSuccess;
  const int smem = BULK ? st.bytes * st.stages : 0;
  auto go = [&](auto kernel, auto... args) {
    cudaError_t e = smem > 40 * 1024 ? ensure_smem((const void *)kernel, BN_SMEM) : cudaSuccess;
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(s.threads), smem, l.stream, a, s.group, st, args...);
  };
  if (l.backward) return go(block_norm_bwd_kernel<TE, TR, VEC, CH, R, BULK>, l.part, l.status);
  return go(block_norm_kernel<TE, TR, VEC, CH, R, BULK>, l.status);
}

template <typename TE, typename TR, int VEC, int CH>
static cudaError_t bn_launch(const BnLaunch &l, const BnShape &s) {
  BnStages st = bn_inputs(l.a, l.backward);
  const int ctas = std::max(1, bn_resident(l.backward, VEC, CH) / s.threads);
  // Several rows a group where registers and shared memory hold them and all CTAs still get two blocks.
  constexpr int R = VEC * CH <= 8 ? 2 : 1;
  if (R > 1 && l.a.T >= (int64_t)device_sms() * ctas * (s.threads / s.group) * R * 2 && bn_stages(l.a, s, ctas, R, st))
    return bn_go<TE, TR, VEC, CH, R, true>(l, s, ctas, st);
  if (bn_stages(l.a, s, ctas, 1, st)) return bn_go<TE, TR, VEC, CH, 1, true>(l, s, ctas, st);
  return bn_go<TE, TR, VEC, CH, 1, false>(l, s, ctas, st);
}

template <typename TE, typename TR>
static cudaError_t bn_dispatch(const BnLaunch &l, const BnShape &s) {
  constexpr int W = Vec16<TE>::N;
  if (s.vec == 1) {
    if (s.ch == 2) return bn_launch<TE, TR, 1, 2>(l, s);
    if (s.ch == 8) return bn_launch<TE, TR, 1, 8>(l, s);
    return bn_launch<TE, TR, 1, 32>(l, s);
  }
  if (s.ch == 1) return bn_launch<TE, TR, W, 1>(l, s);
  if (s.ch == 2) return bn_launch<TE, TR, W, 2>(l, s);
  return bn_launch<TE, TR, W, 32 / W>(l, s);
}

static cudaError_t bn_any(const BnLaunch &l) {
  const BnShape s = bn_shape(l.a);
  if (l.a.f32) return bn_dispatch<float, float>(l, s);
  if (l.a.rf32) return bn_dispatch<__nv_bfloat16, float>(l, s);
  return bn_dispatch<__nv_bfloat16, __nv_bfloat16>(l, s);
}

cudaError_t launch_block_norm(const NormArgs &a, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return bn_any({a, false, nullptr, status, stream, nullptr, false});
}

size_t block_norm_scratch_bytes(const NormArgs &a) {
  if (a.T == 0) return 0;
  int groups = 0;
  bn_any({a, true, nullptr, nullptr, nullptr, &groups, true});
  return (size_t)3 * groups * a.H * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const NormArgs &a, void *scratch, int *status, cudaStream_t stream) {
  float *dg = a.gate_kind == MOE_GATE_CHANNEL ? (float *)a.dgate : nullptr;
  if (a.T == 0) {
    cudaError_t e = cudaSuccess;
    for (float *p : {a.dw_pre, a.dw_post, dg})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)a.H * 4, stream);
    return e;
  }
  int groups = 0;
  cudaError_t e = bn_any({a, true, (float *)scratch, status, stream, &groups, false});
  if (e != cudaSuccess || (!a.dw_pre && !a.dw_post && !dg)) return e;
  return launch_pdl(block_norm_join_kernel, dim3((unsigned)ceil_div(a.H, 32), 3), dim3(32, 32), 0, stream,
                    (const float *)scratch, (int64_t)groups, a.H, a.dw_pre, a.dw_post, dg);
}

}  // namespace moe

// The join between two blocks: norm after a block, gate, scaled residual sum
// and norm before the next block, forward and backward (contracts with
// moe_block_norm in moe.h).
//
// A row belongs to a group of threads, 4 to 32 lanes of a warp for short
// rows and a whole CTA for others, and stays in registers between its loads
// and its stores: every input is read once.  CTAs walk over the rows; the
// inputs of the next few blocks of rows are on their way to shared memory by
// bulk copies meanwhile.  A row that starts between 16-byte boundaries is
// copied with the bytes around it, so odd widths need no loads of their own.
// A group takes two rows at a time where there are enough of them, so that the
// rounds of a sum over a row, which are latency, are shared.  Rows too long
// for two stages are loaded straight from memory.  A row's statistics are
// summed in an order set by H, the load width and, for up to 256 channels,
// whether the inputs are dense, so its outputs do not depend on the other rows.
//
// What it moves is the floor: 29.6 us for the join of 8192 rows of 2048
// (bfloat16 beside a float residual) at the measured copy rate, 158 us for the
// gradient of 32768 rows with an element gate.  Measured: 38.5 us (77 %) and
// 245 us (64 %).  The join loses its start and its last wave.  The gradient
// waits on its two rounds of sums over a row (shuffles, shared memory and, where
// a CTA shares the row, a barrier each), with 16 warps an SM to fill them: its
// issue slots are busy 48 % of the time and memory 43 %, while its stages are
// there in time (300 of a block's 8600 cycles pass at their barrier).  Above
// 4096 channels (8 or 16 pairs a thread) weights do not stay in registers, a
// group takes one row at a time and one CTA fills the SM's registers: at 4096 x
// 5120 ten warps an SM wait for weights and spilled registers, issue slots busy
// 29 %.  Measured on the way for the gradient at 32768 x 2048: row loads without stages 435 us, stages with one row a group
// 367, two 308, weights held and pairs 274, no test a load 244; one row a group
// and five stages 289, three CTAs an SM with fewer registers 307.
//
// Backward: with v = r_out, x = v rstd the normed row and g = dh w,
//   dr = dr_out + rstd g - v c,   c = rstd^3 mean(g v)
// (the derivative of v -> v rsqrt(mean v^2 + eps)), and the same once more for
// y with u = scale gate dr in place of dh.  The row's first round of sums
// (v^2, g v, y^2) gives dr, the second (u w y) gives dy.  The gradients of
// the weights are sums over rows: each group keeps those of its own rows in
// registers, a CTA writes those of its groups once, and a second kernel adds the
// CTAs in order.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int BN_MAX_THREADS = 512, BN_MAX_STAGES = 6, BN_MAX_INPUTS = 5;

// The row inputs of a launch (NULL: not there) and where their blocks of rows
// stand in a stage.  Forward: r, y, element gate; backward: dr_out, r_out, dh,
// y, element gate.
struct BnStages {
  int n, stages, bytes;  // inputs, stages, bytes of a stage
  int rows;              // of a block
  int runs;              // runs of bytes that it is: 1 (rows behind one another), or its rows
  int near;              // rows that may start within 16 bytes of an input's start, or end within 16 of its end
  int off[BN_MAX_INPUTS], es[BN_MAX_INPUTS];
  uint32_t row[BN_MAX_INPUTS];    // bytes from row to row in a stage
  uint32_t apart[BN_MAX_INPUTS];  // and in memory (modulo 2^32)
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
  if (first_row >= T || !st.base[k]) return p;
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
    umma::bulk_load(stage + st.off[k] + q * st.row[k] + (p.from - (p.lo & ~(uintptr_t)15)), (const void *)p.from, bytes, bar);
}
// What the copies of a block may have missed (the whole CTA; the caller's
// barrier follows): bytes of the pieces that an input starts or ends in, in
// which only the first and the last `near` rows lie.  ZERO: rows of the last
// block that the inputs lack are zeros.
template <bool ZERO>
__device__ inline bool bn_mend(const BnStages &st, uint8_t *stage, int64_t t0, int T, int H) {
  if (t0 >= st.near && t0 + st.rows + st.near <= T) return false;
  bool missed = false;
  for (int k = 0; k < st.n; ++k)
    for (int q = 0; q < st.runs; ++q) {
      const BnPiece p = bn_piece(st, k, q, t0, T, H);
      if (p.from <= p.lo && p.to >= p.hi) continue;
      missed = true;
      uint8_t *dst = stage + st.off[k] + q * st.row[k] - (p.lo & ~(uintptr_t)15);
      for (uintptr_t b = p.lo + threadIdx.x; b < p.hi; b += blockDim.x)
        if (b < p.from || b >= p.to) dst[b] = *(const uint8_t *)b;
    }
  if (ZERO && t0 + st.rows > T) {
    const int rows = (int)(T - t0);
    for (int k = 0; k < st.n; ++k) {
      if (!st.base[k]) continue;
      uint8_t *row = stage + st.off[k] + rows * st.row[k];
      if (st.runs == 1) row += ((uintptr_t)st.base[k] + t0 * st.ld[k] * st.es[k]) & 15;
      for (uint32_t b = 2 * threadIdx.x; b < (st.rows - rows) * st.row[k]; b += 2 * blockDim.x) *(uint16_t *)(row + b) = 0;
    }
    missed = true;
  }
  // The stage is copied to again later; without this a copy may pass these writes.
  if (missed) umma::fence_proxy_async_smem();
  return missed;
}

// ---- what a thread holds of a row: NP pairs of floats ----
// Wide: CH runs of VEC neighbouring elements, at (c group + lane) VEC.  Scalar
// (VEC = 1): elements lane, lane + group, ...  Past the row it holds zeros;
// FULL: no thread reaches past the row.
template <int VEC, int CH, bool FULL>
struct BnRow {
  static constexpr int NP = VEC * CH / 2;
  int lane, group, H;

  template <typename T>
  __device__ inline void load(const T *row, F2 (&o)[NP]) const {
    if constexpr (VEC == 1) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = 2 * p * group + lane;
        o[p] = F2(i < H ? Elem<T>::load(row + i) : 0.f, i + group < H ? Elem<T>::load(row + i + group) : 0.f);
      }
    } else {
      constexpr int N = Vec16<T>::N;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
#pragma unroll
        for (int b = 0; b < VEC / N; ++b) {
          float v[N];
          uint4 raw = {0, 0, 0, 0};
          if (FULL || i < H) raw = *(const uint4 *)(row + i + b * N);
          Vec16<T>::unpack(raw, v);
#pragma unroll
          for (int k = 0; k < N; k += 2) o[(c * VEC + b * N + k) / 2] = F2(v[k], v[k + 1]);
        }
      }
    }
  }
  template <typename T>
  __device__ inline void store(T *row, const F2 (&x)[NP]) const {
    if constexpr (VEC == 1) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = 2 * p * group + lane;
        float a, b;
        x[p].get(a, b);
        if (i < H) row[i] = Elem<T>::from_f32(a);
        if (i + group < H) row[i + group] = Elem<T>::from_f32(b);
      }
    } else {
      constexpr int N = Vec16<T>::N;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * group + lane) * VEC;
#pragma unroll
        for (int b = 0; b < VEC / N; ++b) {
          float v[N];
#pragma unroll
          for (int k = 0; k < N; k += 2) x[(c * VEC + b * N + k) / 2].get(v[k], v[k + 1]);
          if (FULL || i < H) Vec16<T>::store(row + i + b * N, v);
        }
      }
    }
  }
  // Weights and channel gates: float or the rows' type.
  template <typename T>
  __device__ inline void weights(const void *p, bool f32, float add, F2 (&o)[NP]) const {
    if (f32) load((const float *)p, o);
    else load((const T *)p, o);
#pragma unroll
    for (int k = 0; k < NP; ++k) o[k] = add2(o[k], F2(add));
  }
};

// Sums of N values (at most 8) over the threads of a row, in a fixed order; all
// get them.  A warp halves the number of values that a lane holds as it halves
// the lanes that a value is spread over; the sums of several warps meet in
// `buf`, where a quarter of a value's slots goes to each of four lanes (slots
// past the last warp hold zeros).  Consecutive calls alternate between two
// buffers: the barrier of one call tells that the buffer of the call before it
// has been read.
template <int N>
__device__ inline void bn_row_sum(float (&v)[N], int group, float (*buf)[16]) {
  static_assert(N <= 8, "a value's quarter for each lane");
  const int lane = threadIdx.x & 31;
  if (group < 32) {
    for (int d = group >> 1; d; d >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(FULL_MASK, v[n], d);
    return;
  }
  constexpr int H1 = (N + 1) / 2, H2 = (H1 + 1) / 2, H3 = (H2 + 1) / 2;
  float x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = v[n];
  auto halve = [&](auto count, auto half, int d) {
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < half.value; ++i) {
      if (i + half.value < count.value) {
        const float send = upper ? x[i] : x[i + half.value], keep = upper ? x[i + half.value] : x[i];
        x[i] = keep + __shfl_xor_sync(FULL_MASK, send, d);
      } else {  // no partner: a plain sum, which both sides hold
        x[i] += __shfl_xor_sync(FULL_MASK, x[i], d);
      }
    }
  };
  halve(std::integral_constant<int, N>(), std::integral_constant<int, H1>(), 16);
  halve(std::integral_constant<int, H1>(), std::integral_constant<int, H2>(), 8);
  halve(std::integral_constant<int, H2>(), std::integral_constant<int, H3>(), 4);
  x[0] += __shfl_xor_sync(FULL_MASK, x[0], 2);
  x[0] += __shfl_xor_sync(FULL_MASK, x[0], 1);
  // The lane that holds value n.
  auto holder = [](int n) {
    int l = 0;
    if (N > 1 && n >= H1) n -= H1, l |= 16;
    if (H1 > 1 && n >= H2) n -= H2, l |= 8;
    if (H2 > 1 && n >= H3) n -= H3, l |= 4;
    return l;
  };
  if (group == 32) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = __shfl_sync(FULL_MASK, x[0], holder(n));
    return;
  }
  // (a lane without a value of its own holds a copy of another one's)
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane == holder(n)) buf[n][warp] = x[0];
  __syncthreads();
  float s = 0.f;
  if (lane < 4 * N) {
    const float4 f = *(const float4 *)&buf[lane >> 2][4 * (lane & 3)];
    s = (f.x + f.y) + (f.z + f.w);
  }
  s += __shfl_xor_sync(FULL_MASK, s, 1);
  s += __shfl_xor_sync(FULL_MASK, s, 2);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = __shfl_sync(FULL_MASK, s, 4 * n);
}

// A wait ran out and the CTA ends: its copies in flight land first, those of
// the block in `slot` and of the blocks behind it (or a limit passes for each
// stage that has none).
static __device__ __noinline__ void bn_drain(BnBars &bars, int stages, int slot, uint32_t phase) {
  for (int i = 0; i < stages; ++i) {
    umma::mbar_drain(&bars.full[slot], phase);
    if (++slot == stages) slot = 0, phase ^= 1;
  }
}

// A CTA's walk over its blocks of rows, with stages (BULK) or without.
template <bool BULK, int R, bool ZERO>
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
    bool ok = umma::mbar_wait(&bars.full[slot], phase, &bars.abort_flag, status);
    // (the gradient's lanes leave together: it runs 1 to 5 % faster with the vote,
    // the join of odd rows 5 % slower)
    if (ZERO) ok = __all_sync(FULL_MASK, ok);
    if (!ok) {
      bn_drain(bars, st.stages, slot, phase);
      return false;
    }
    if (bn_mend<ZERO>(st, stage, t0, T, H)) __syncthreads();
    return true;
  }
  // Row `at` of the block (row t in memory, of `p`) of input K.
  template <int K, bool WIDE, typename E>
  __device__ inline const E *row(const void *p, int64_t ld, int64_t t, int at) const {
    if (!BULK) return (const E *)p + t * ld;
    uint32_t o = st.off[K] + at * st.row[K];
    // where the run starts between 16-byte boundaries
    if (!WIDE) o += ((uint32_t)(uintptr_t)st.base[K] + (uint32_t)(st.runs > 1 ? t : t0) * st.apart[K]) & 15;
    return (const E *)(stage + o);
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
constexpr int bn_resident(bool backward, int np, int r) { return !backward && np <= 4 && r == 1 ? 1024 : 512; }

// An output's rows: row j of a group in a block, by a pointer that moves on.
template <typename E>
struct BnOut {
  E *p;
  int64_t next, step;  // elements from row j to j + 1, and to the next block
  __device__ inline BnOut(void *base, int64_t ld, int64_t t, int per_cta, int64_t step_rows)
      : p((E *)base + t * ld), next(per_cta * ld), step(step_rows * ld) {}
  __device__ inline E *row(int j) const { return p + j * next; }
  __device__ inline void move() { p += step; }
};

// The rows of a block that a group takes: number, place in the block, whether
// there is such a row.  Where there is none, the block's first row stands in
// or, with ZERO, a row of zeros.
template <int R, bool ZERO>
struct BnRows {
  int64_t t[R];
  int at[R];
  bool there[R];
  __device__ inline BnRows(int64_t t0, int per_cta, int sub, int T) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      there[j] = t0 + j * per_cta + sub < T;
      at[j] = ZERO || there[j] ? j * per_cta + sub : 0;
      t[j] = there[j] ? t0 + at[j] : t0;
    }
  }
};

template <typename TE, typename TR, int VEC, int CH, int R, bool BULK, bool FULL>
__global__ void __launch_bounds__(BN_MAX_THREADS, bn_resident(false, VEC * CH / 2, R) / BN_MAX_THREADS)
block_norm_kernel(const NormArgs a, int group, const BnStages st, int *status) {
  constexpr int NP = VEC * CH / 2;
  constexpr bool WIDE = VEC > 1, HELD = NP <= 4;  // weights stay in registers
  extern __shared__ __align__(128) uint8_t bn_smem[];
  __shared__ BnBars bars;
  __shared__ __align__(16) float buf[2][R][16];
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  const BnRow<VEC, CH, FULL> io = {lane, group, a.H};
  if (threadIdx.x < 2 * R * 16) buf[0][0][threadIdx.x] = 0.f;
  if (!BULK) __syncthreads();
  BnWalk<BULK, R, false> walk(st, a.T, a.H, per_cta, bn_smem, bars);
  BnOut<TR> r_out(a.r_out, a.ld_r_out, walk.t0 + sub, per_cta, walk.step);
  BnOut<TE> h_out(a.h, a.ld_h, walk.t0 + sub, per_cta, walk.step);
  F2 w_post[NP], w_pre[NP];
  if (HELD && a.w_post) io.template weights<TE>(a.w_post, a.wf32, a.offset, w_post);
  if (HELD && a.w_pre) io.template weights<TE>(a.w_pre, a.wf32, a.offset, w_pre);
  int round = 0;
  for (; walk.t0 < a.T; walk.next()) {
    if (!walk.arrive(status)) return;
    const BnRows<R, false> rows(walk.t0, per_cta, sub, a.T);
    float s[R], rstd[R];
    F2 v[R][NP], y[NP];
#pragma unroll
    for (int j = 0; j < R; ++j) rstd[j] = 1.f;
    if (a.w_post) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        io.load(walk.template row<1, WIDE, TE>(a.y, a.ld_y, rows.t[j], rows.at[j]), y);
        F2 sum(0.f);
#pragma unroll
        for (int p = 0; p < NP; ++p) sum = fma2(y[p], y[p], sum);
        s[j] = sum.sum();
      }
      bn_row_sum(s, group, buf[round++ & 1]);
#pragma unroll
      for (int j = 0; j < R; ++j) rstd[j] = rsqrtf(fmaf(s[j], inv_h, a.eps));
    }
    if (BULK && (!a.w_post || group <= 32)) __syncthreads();
    walk.refill();
    if (!HELD && a.w_post) io.template weights<TE>(a.w_post, a.wf32, a.offset, w_post);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t t = rows.t[j];
      io.load(walk.template row<0, WIDE, TR>(a.r, a.ld_r, t, rows.at[j]), v[j]);
      if (a.y) {
        io.load(walk.template row<1, WIDE, TE>(a.y, a.ld_y, t, rows.at[j]), y);
        const F2 f(a.w_post ? a.scale * rstd[j] : a.scale);
#pragma unroll
        for (int p = 0; p < NP; ++p) y[p] = mul2(y[p], f);
        if (a.w_post) {
#pragma unroll
          for (int p = 0; p < NP; ++p) y[p] = mul2(y[p], w_post[p]);
        }
        F2 g[NP];
        if (a.gate_kind == MOE_GATE_ELEMENT) io.load(walk.template row<2, WIDE, TE>(a.gate, a.ld_gate, t, rows.at[j]), g);
        else if (a.gate_kind == MOE_GATE_CHANNEL) io.template weights<TE>(a.gate, a.wf32, 0.f, g);
        else {
          const F2 one(a.gate_kind == MOE_GATE_TOKEN ? ((const float *)a.gate)[t] : 1.f);
#pragma unroll
          for (int p = 0; p < NP; ++p) g[p] = one;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) v[j][p] = fma2(g[p], y[p], v[j][p]);
        if (rows.there[j]) io.store(r_out.row(j), v[j]);
      }
      F2 sum(0.f);
#pragma unroll
      for (int p = 0; p < NP; ++p) sum = fma2(v[j][p], v[j][p], sum);
      s[j] = sum.sum();
    }
    if (a.w_pre) {
      bn_row_sum(s, group, buf[round++ & 1]);
      if (!HELD) io.template weights<TE>(a.w_pre, a.wf32, a.offset, w_pre);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const F2 rs(rsqrtf(fmaf(s[j], inv_h, a.eps)));
#pragma unroll
        for (int p = 0; p < NP; ++p) v[j][p] = mul2(mul2(v[j][p], rs), w_pre[p]);
        if (rows.there[j]) io.store(h_out.row(j), v[j]);
      }
    }
    r_out.move();
    h_out.move();
  }
}

// part: [3][CTAs][H] sums over a CTA's rows of what dw_pre, dw_post and a channel
// gate's gradient are made of (only those that the call asks for).
template <typename TE, typename TR, int VEC, int CH, int R, bool BULK, bool FULL>
__global__ void __launch_bounds__(BN_MAX_THREADS)
block_norm_bwd_kernel(const NormArgs a, int group, const BnStages st, float *part, int *status) {
  constexpr int NP = VEC * CH / 2;
  constexpr bool WIDE = VEC > 1, HELD = NP <= 4;
  extern __shared__ __align__(128) uint8_t bn_smem[];
  __shared__ BnBars bars;
  __shared__ __align__(16) float buf[2][3 * R][16];
  const int per_cta = blockDim.x / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const float inv_h = 1.f / a.H;
  const BnRow<VEC, CH, FULL> io = {lane, group, a.H};
  for (int i = threadIdx.x; i < 2 * 3 * R * 16; i += blockDim.x) buf[0][0][i] = 0.f;
  if (!BULK) __syncthreads();
  BnWalk<BULK, R, true> walk(st, a.T, a.H, per_cta, bn_smem, bars);
  BnOut<TR> dr_out(a.dr, a.ld_dr, walk.t0 + sub, per_cta, walk.step);
  BnOut<TE> dy_out(a.dy, a.ld_dy, walk.t0 + sub, per_cta, walk.step), dg_out(a.dgate, a.ld_dgate, walk.t0 + sub, per_cta, walk.step);
  F2 w_post[NP], w_pre[NP], dw_post[NP], dw_pre[NP], dgate[NP];
  if (HELD && a.w_post) io.template weights<TE>(a.w_post, a.wf32, a.offset, w_post);
  if (HELD && a.w_pre) io.template weights<TE>(a.w_pre, a.wf32, a.offset, w_pre);
#pragma unroll
  for (int p = 0; p < NP; ++p) dw_post[p] = dw_pre[p] = dgate[p] = F2(0.f);
  int round = 0;
  for (; walk.t0 < a.T; walk.next()) {
    if (!walk.arrive(status)) return;
    const BnRows<R, true> rows(walk.t0, per_cta, sub, a.T);
    float s[3 * R];  // v^2, dh w v, y^2 of each row
    if (!HELD && a.w_pre) io.template weights<TE>(a.w_pre, a.wf32, a.offset, w_pre);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      F2 vv(0.f), dv(0.f), yy(0.f), x[NP], d[NP];
      if (a.w_pre) {
        io.load(walk.template row<1, WIDE, TR>( a.r_out, a.ld_r_out, rows.t[j], rows.at[j]), x);
        io.load(walk.template row<2, WIDE, TE>( a.dh, a.ld_dh, rows.t[j], rows.at[j]), d);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          vv = fma2(x[p], x[p], vv);
          dv = fma2(mul2(d[p], w_pre[p]), x[p], dv);
        }
      }
      if (a.w_post) {
        io.load(walk.template row<3, WIDE, TE>( a.y, a.ld_y, rows.t[j], rows.at[j]), x);
#pragma unroll
        for (int p = 0; p < NP; ++p) yy = fma2(x[p], x[p], yy);
      }
      s[3 * j] = vv.sum();
      s[3 * j + 1] = dv.sum();
      s[3 * j + 2] = yy.sum();
    }
    bn_row_sum(s, group, buf[round++ & 1]);
    if (BULK && group <= 32) __syncthreads();
    walk.refill();
    if (!HELD && a.w_post) io.template weights<TE>(a.w_post, a.wf32, a.offset, w_post);
    float ry[R], q[2 * R];  // q: u w y, scale dr w y
    F2 e[R][NP];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t t = rows.t[j];
      // A row of zeros in the place of one that is not there adds nothing to
      // the sums over rows: with factors of zero not even where eps is 0.
      const bool in = rows.there[j];
      const float rv = in ? rsqrtf(fmaf(s[3 * j], inv_h, a.eps)) : 0.f;
      ry[j] = !in ? 0.f : a.w_post ? rsqrtf(fmaf(s[3 * j + 2], inv_h, a.eps)) : 1.f;
      if (a.dr_out) {
        io.load(walk.template row<0, WIDE, TR>(a.dr_out, a.ld_dr_out, t, rows.at[j]), e[j]);
      } else {
#pragma unroll
        for (int p = 0; p < NP; ++p) e[j][p] = F2(0.f);
      }
      if (a.w_pre) {
        F2 x[NP], d[NP];
        io.load(walk.template row<1, WIDE, TR>( a.r_out, a.ld_r_out, t, rows.at[j]), x);
        io.load(walk.template row<2, WIDE, TE>( a.dh, a.ld_dh, t, rows.at[j]), d);
        const F2 rr(rv), cr(-(s[3 * j + 1] * inv_h * rv * rv * rv));
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          dw_pre[p] = fma2(d[p], mul2(x[p], rr), dw_pre[p]);
          e[j][p] = add2(e[j][p], fma2(mul2(d[p], w_pre[p]), rr, mul2(x[p], cr)));
        }
        if (rows.there[j]) io.store(dr_out.row(j), e[j]);
      }
      q[2 * j] = q[2 * j + 1] = 0.f;
      if (a.y) {
        F2 y[NP], g[NP], q0(0.f), q1(0.f);
        io.load(walk.template row<3, WIDE, TE>( a.y, a.ld_y, t, rows.at[j]), y);
        const F2 sc(a.scale), rr(ry[j]);
#pragma unroll
        for (int p = 0; p < NP; ++p) e[j][p] = mul2(e[j][p], sc);
        if (a.gate_kind != MOE_GATE_NONE) {
          if (a.gate_kind == MOE_GATE_ELEMENT) io.load(walk.template row<4, WIDE, TE>( a.gate, a.ld_gate, t, rows.at[j]), g);
          else if (a.gate_kind == MOE_GATE_CHANNEL) io.template weights<TE>(a.gate, a.wf32, 0.f, g);
          else {
            const F2 gt(in ? ((const float *)a.gate)[t] : 0.f);
#pragma unroll
            for (int p = 0; p < NP; ++p) g[p] = gt;
          }
          // the gate's gradient, and u in the place of scale dr
          F2 dg[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            dg[p] = mul2(e[j][p], mul2(y[p], rr));
            if (a.w_post) dg[p] = mul2(dg[p], w_post[p]);
            q1 = add2(q1, dg[p]);
            e[j][p] = mul2(e[j][p], g[p]);
          }
          if (a.gate_kind == MOE_GATE_CHANNEL) {
#pragma unroll
            for (int p = 0; p < NP; ++p) dgate[p] = add2(dgate[p], dg[p]);
          }
          if (a.gate_kind == MOE_GATE_ELEMENT && rows.there[j]) io.store(dg_out.row(j), dg);
        }
        if (a.w_post) {
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const F2 x = mul2(y[p], rr);
            dw_post[p] = fma2(e[j][p], x, dw_post[p]);
            e[j][p] = mul2(e[j][p], w_post[p]);
            q0 = fma2(e[j][p], y[p], q0);
            e[j][p] = mul2(e[j][p], rr);  // dy but for its last term
          }
        }
        q[2 * j] = q0.sum();
        q[2 * j + 1] = q1.sum();
      }
    }
    if (a.y) {
      if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) bn_row_sum(q, group, buf[round++ & 1]);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (a.gate_kind == MOE_GATE_TOKEN && lane == 0 && rows.there[j]) ((float *)a.dgate)[rows.t[j]] = q[2 * j + 1];
        if (a.w_post) {
          const F2 cy(-(q[2 * j] * inv_h * ry[j] * ry[j] * ry[j]));
          F2 y[NP];
          io.load(walk.template row<3, WIDE, TE>( a.y, a.ld_y, rows.t[j], rows.at[j]), y);
#pragma unroll
          for (int p = 0; p < NP; ++p) e[j][p] = fma2(y[p], cy, e[j][p]);
        }
        if (rows.there[j]) io.store(dy_out.row(j), e[j]);
      }
    }
    dr_out.move();
    dy_out.move();
    dg_out.move();
  }
  // The groups of a CTA as one: lanes, then warps, in a fixed order.
  float *p = part + (int64_t)blockIdx.x * a.H;
  const int64_t apart = (int64_t)gridDim.x * a.H;
  auto leave = [&](F2 (&x)[NP], float *out) {
    if (NP <= 4 && per_cta > 1) {
      const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
      float *red = (float *)bn_smem;  // [warps][H]: the stages are done with
      for (int d = group; d < 32; d <<= 1) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          float u, v;
          x[q].get(u, v);
          u += __shfl_xor_sync(FULL_MASK, u, d);
          v += __shfl_xor_sync(FULL_MASK, v, d);
          x[q] = F2(u, v);
        }
      }
      __syncthreads();
      if ((threadIdx.x & 31) < group) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          float u, v;
          x[q].get(u, v);
          const int i = ((2 * q) / VEC * group + lane) * VEC + (2 * q) % VEC, k = VEC == 1 ? i + group : i + 1;
          if (i < a.H) red[warp * a.H + i] = u;
          if (k < a.H) red[warp * a.H + k] = v;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float sum = 0.f;
        for (int w = 0; w < warps; ++w) sum += red[w * a.H + i];
        out[i] = sum;
      }
    } else {
      io.store(out, x);
    }
  };
  if (a.dw_pre) leave(dw_pre, p);
  if (a.dw_post) leave(dw_post, p + apart);
  if (a.gate_kind == MOE_GATE_CHANNEL) leave(dgate, p + 2 * apart);
}

// ---------------------------------------------------------------- host
// Load width; pairs of elements a thread; threads of a row (a power of two up to
// 32, or a multiple of 32); threads of a CTA.
struct BnShape {
  int vec, pairs, group, threads;
};

inline bool bn_wide(const NormArgs &a, int vec) {
  auto row = [&](const void *p, int64_t ld, int es) { return !p || (((uintptr_t)p & 15) == 0 && ld * es % 16 == 0); };
  const int e = a.f32 ? 4 : 2, r = a.rf32 ? 4 : 2;
  bool ok = a.H % vec == 0 && row(a.r, a.ld_r, r) && row(a.y, a.ld_y, e) && row(a.r_out, a.ld_r_out, r) &&
            row(a.h, a.ld_h, e) && row(a.dr_out, a.ld_dr_out, r) && row(a.dh, a.ld_dh, e) && row(a.dr, a.ld_dr, r) &&
            row(a.dy, a.ld_dy, e) && row(a.w_post, 0, 1) && row(a.w_pre, 0, 1);
  if (a.gate_kind == MOE_GATE_CHANNEL) ok = ok && row(a.gate, 0, 1);
  if (a.gate_kind == MOE_GATE_ELEMENT) ok = ok && row(a.gate, a.ld_gate, e) && row(a.dgate, a.ld_dgate, e);
  return ok;
}

// All but the load width.  dense: the rows of every input stand behind one another.
inline BnShape bn_threads(int H, bool dense) {
  BnShape s;
  s.vec = 0;
  s.pairs = 4;
  while (s.pairs < 16 && ceil_div(H, 2 * s.pairs) > BN_MAX_THREADS) s.pairs *= 2;
  const int need = (int)ceil_div(H, 2 * s.pairs);
  if (need <= 32) {
    s.group = 4;
    while (s.group < need) s.group *= 2;
    s.threads = 256;
    if (!dense) s.threads = s.group = 32;  // one row a CTA: its inputs are copied row by row
  } else {
    s.group = (int)round_up(need, 32);
    s.threads = s.group;
  }
  return s;
}
inline BnShape bn_shape(const NormArgs &a, bool dense) {
  BnShape s = bn_threads(a.H, dense);
  s.vec = a.f32 ? 4 : 8;
  if (!bn_wide(a, s.vec)) s.vec = 1;
  return s;
}
// CTAs of an SM, where a group takes r rows at a time.
inline int bn_ctas(bool backward, const BnShape &s, int r) { return std::max(1, bn_resident(backward, s.pairs, r) / s.threads); }

// The most CTAs that a gradient's launch has, whichever of its inputs are
// there: their strides alone tell (where all are dense, those given are).
inline int64_t bn_most_ctas(const NormArgs &a) {
  bool dense = true;
  for (int64_t ld : {a.ld_dr_out, a.ld_r_out, a.ld_dh, a.ld_y, a.ld_gate}) dense = dense && ld == a.H;
  int64_t most = 0;
  for (bool d : {true, dense}) {
    const BnShape s = bn_threads(a.H, d);
    most = std::max(most, std::min(ceil_div(a.T, s.threads / s.group), (int64_t)device_sms() * bn_ctas(true, s, 1)));
  }
  return most;
}

// The inputs that rows come from, in the order in which the kernels name them.
inline BnStages bn_inputs(const NormArgs &a, bool backward) {
  BnStages st = {};
  const int e = a.f32 ? 4 : 2, r = a.rf32 ? 4 : 2;
  auto add = [&](const void *p, int64_t ld, int es) {
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
inline bool bn_stages(const NormArgs &a, const BnShape &s, int ctas, int R, BnStages &st) {
  const int per_cta = s.threads / s.group;
  st.rows = per_cta * R;
  st.runs = st.near = 1;
  st.bytes = 0;
  for (int k = 0; k < st.n; ++k)
    if (st.base[k] && st.rows > 1 && st.ld[k] != a.H) st.runs = st.rows;
  if (st.runs > 1 && (per_cta > 1 || st.runs * st.n > 32)) return false;
  for (int k = 0; k < st.n; ++k) {
    if (!st.base[k]) continue;
    const int run = (int)round_up((int64_t)(st.runs > 1 ? 1 : st.rows) * a.H * st.es[k], 16) + 16;
    st.off[k] = st.bytes;
    st.row[k] = st.runs > 1 ? run : a.H * st.es[k];
    st.apart[k] = (uint32_t)(st.ld[k] * st.es[k]);
    st.near = std::max(st.near, (int)ceil_div(16, st.ld[k] * st.es[k]));
    st.bytes += st.runs * run;
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
  int *groups;  // out: CTAs, each of which leaves partial sums
};

template <typename TE, typename TR, int VEC, int CH, int R, bool BULK, bool FULL = false>
static cudaError_t bn_go(const BnLaunch &l, const BnShape &s, int ctas, const BnStages &st) {
  const NormArgs &a = l.a;
  const int per_cta = s.threads / s.group;
  const int grid = (int)std::min<int64_t>(ceil_div(a.T, per_cta * R), (int64_t)device_sms() * ctas);
  if (l.groups) *l.groups = grid;
  const int smem = BULK ? st.bytes * st.stages : 0;
  auto go = [&](auto kernel, auto... args) {
    cudaError_t e = smem > 40 * 1024 ? ensure_smem((const void *)kernel, BN_SMEM) : cudaSuccess;
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(s.threads), smem, l.stream, a, s.group, st, args...);
  };
  if (l.backward) return go(block_norm_bwd_kernel<TE, TR, VEC, CH, R, BULK, FULL>, l.part, l.status);
  return go(block_norm_kernel<TE, TR, VEC, CH, R, BULK, FULL>, l.status);
}

template <typename TE, typename TR, int VEC, int NP>
static cudaError_t bn_launch(const BnLaunch &l, const BnShape &s) {
  constexpr int CH = 2 * NP / VEC;
  BnStages st = bn_inputs(l.a, l.backward);
  int ctas = bn_ctas(l.backward, s, 2);
  if constexpr (NP <= 4) {
    const bool full = VEC > 1 && l.a.H == s.group * VEC * CH;
    // Two rows a group where shared memory holds them and all CTAs still get two blocks.
    if (l.a.T >= (int64_t)device_sms() * ctas * (s.threads / s.group) * 4 && bn_stages(l.a, s, ctas, 2, st)) {
      if constexpr (VEC > 1)
        if (full) return bn_go<TE, TR, VEC, CH, 2, true, true>(l, s, ctas, st);
      return bn_go<TE, TR, VEC, CH, 2, true>(l, s, ctas, st);
    }
    ctas = bn_ctas(l.backward, s, 1);
    if (!bn_stages(l.a, s, ctas, 1, st)) return cudaErrorInvalidConfiguration;  // (at most 4096 elements: they fit)
    if constexpr (VEC > 1)
      if (full) return bn_go<TE, TR, VEC, CH, 1, true, true>(l, s, ctas, st);
    return bn_go<TE, TR, VEC, CH, 1, true>(l, s, ctas, st);
  } else {
    if (bn_stages(l.a, s, ctas, 1, st)) return bn_go<TE, TR, VEC, CH, 1, true>(l, s, ctas, st);
    return bn_go<TE, TR, VEC, CH, 1, false>(l, s, ctas, st);
  }
}

template <typename TE, typename TR>
cudaError_t bn_dispatch(const BnLaunch &l) {
  constexpr int W = Vec16<TE>::N;
  bool dense = true;
  const BnStages st = bn_inputs(l.a, l.backward);
  for (int k = 0; k < st.n; ++k) dense = dense && (!st.base[k] || st.ld[k] == l.a.H);
  const BnShape s = bn_shape(l.a, dense);
  if (s.vec == 1) {
    if (s.pairs == 4) return bn_launch<TE, TR, 1, 4>(l, s);
    if (s.pairs == 8) return bn_launch<TE, TR, 1, 8>(l, s);
    return bn_launch<TE, TR, 1, 16>(l, s);
  }
  if (s.pairs == 4) return bn_launch<TE, TR, W, 4>(l, s);
  if (s.pairs == 8) return bn_launch<TE, TR, W, 8>(l, s);
  return bn_launch<TE, TR, W, 16>(l, s);
}

}  // namespace moe

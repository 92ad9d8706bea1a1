// Cross entropy of the next token from hidden rows: the rows that count, the
// join of the tiles' statistics, and the order of the launches.
//
//   x = scale h W^T    lse = log sum exp x    loss = lse - x[target] + z lse^2
//   g = scale dloss ((1 + 2 z lse) exp(x - lse) - onehot)    dh = g W    dW = g^T h
//
// Rows that count are copied together first, in order: rows that are left out
// cost nothing afterwards, what they hold reaches no product, and the copies
// have the alignment that the tensor maps want whatever the caller's have.
// Then one product leaves a maximum and a sum of exponentials for each row and
// 64 columns (8 bytes for 128 of logits), which are joined per row; the
// gradient recomputes the logits a piece of the vocabulary at a time (2 TDV of
// its 6, of a step's 8; keeping them would take 4 TV bytes) and takes
// both products of the piece while it is near L2's size.
//
// The kernels here move little and are bound by latency, at large sizes by
// memory: 5 rows x 2048 x 32000 spend 9 of their 31 us in them and in starts; 4096 x 2048
// rows are copied in 13 us, their statistics over 24576 columns joined in 22
// and the planes of three chunks added in 25 (under ncu, from a cold L2).
#include <math.h>

#include "linear_ce.h"

namespace moe {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.693147180559945309417f;

// ------------------------------------------------------------- which rows count
// One CTA, for more than CE_FUSE rows: place[t] is row t's place among those
// that count (-1: left out), row_of the reverse; the order is kept.
template <typename Id>
__global__ void __launch_bounds__(1024)
ce_places_kernel(int T, int V, int64_t ignore, const Id *targets, int *count, int *row_of, int *place, CeRow *rows,
                 float *loss, float *lse, int *status) {
  griddep_launch();
  griddep_wait();
  constexpr int M = 8;  // rows of a thread at a time, 1024 apart: their loads are in flight together
  __shared__ int sums[M * 32 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += M * 1024) {
    int64_t id[M];
    unsigned vote[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int t = t0 + j * 1024 + threadIdx.x;
      id[j] = t < T ? (int64_t)targets[t] : ignore;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int t = t0 + j * 1024 + threadIdx.x;
      const bool in = id[j] >= 0 && id[j] < V;
      if (!in && id[j] != ignore) record_status(status, STATUS_BAD_TARGET);
      vote[j] = __ballot_sync(FULL_MASK, t < T && in && id[j] != ignore);
      if (lane == 0) sums[j * 32 + warp] = __popc(vote[j]);
    }
    __syncthreads();
    if (warp == 0) {  // the sums before each warp's, in the order of the rows: eight of them a lane
      int own[M], all = 0;
#pragma unroll
      for (int j = 0; j < M; ++j) {
        own[j] = all;
        all += sums[lane * M + j];
      }
      int s = all;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, s, d);
        if (lane >= d) s += o;
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < M; ++j) sums[lane * M + j] = s - all + own[j];
      if (lane == 31) sums[M * 32] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int t = t0 + j * 1024 + threadIdx.x;
      if (t >= T) break;
      const bool keep = vote[j] >> lane & 1;
      const int at = base + sums[j * 32 + warp] + __popc(vote[j] & lanemask_lt());
      place[t] = keep ? at : -1;
      if (keep) {
        row_of[at] = t;
        rows[at].target = (int)id[j];
      } else {
        if (loss) loss[t] = 0.f;
        if (lse) lse[t] = 0.f;
      }
    }
    base += sums[M * 32];
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base;
  // The padding of the last row tile.
  const int end = (int)round_up(base, CE_ROWS);
  for (int i = base + threadIdx.x; i < end; i += 1024) rows[i] = CeRow{0.f, 0.f, 0.f, -1};
}

// What the gradient needs of a row: d = scale * dloss, l its lse, nll = l -
// x[target].  The target's entry is d (p - 1 + 2 z l p); p - 1 by expm1, which
// keeps the bits that nll has: those of its size from the statistics (a step),
// those of l's size where nll is a difference from l (the gradient alone).
// Returns 1 / the row's factor.
template <typename E>
__device__ inline float grad_row(CeRow &r, float d, float l, float nll, float z) {
  const float zl = 2.f * z * l, p = expf(-nll);
  const float g = d * fmaf(zl, p, expm1f(-nll));
  float c = d * (1.f + zl), b = g, inv = 1.f;
  if (sizeof(E) == 2) {
    b = Elem<E>::to_f32(Elem<E>::from_f32(g));
    if (fabsf(g) > 1e-30f && fabsf(b) < 1e38f) {
      inv = g / b;
      c *= b / g;
    }
  }
  r.lse2 = l * LOG2E;
  r.c = c;
  r.b = b;
  return inv;
}

// One row to its place: D elements times f, zeros up to dp.  wide: units of 16 bytes.
template <typename E, bool SCALED>
__device__ inline void put_row(E *dst, const E *src, int D, int64_t dp, float f, bool wide, int lane) {
  constexpr int N = Vec16<E>::N;
  if (wide) {
    const int nu = src ? D / N : 0;
    for (int u = lane; u < (int)(dp / N); u += 32) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (u < nu) {
        w = ((const uint4 *)src)[u];
        if (SCALED) {
          float x[N];
          Vec16<E>::unpack(w, x);
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] *= f;
          Vec16<E>::store(dst + u * N, x);
          continue;
        }
      }
      ((uint4 *)dst)[u] = w;
    }
  } else {
    for (int c = lane; c < (int)dp; c += 32) {
      E x = src && c < D ? src[c] : Elem<E>::from_f32(0.f);
      if (SCALED) x = Elem<E>::from_f32(Elem<E>::to_f32(x) * f);
      dst[c] = x;
    }
  }
}

// Up to this many rows each CTA of ce_rows_kernel counts the rows before its
// own by itself: reading all targets again costs less than a launch.
constexpr int CE_FUSE = 4096;

// A warp a row: the rows that count to their places, zeros behind them (in
// the columns up to dp and the rows up to the tile's end), zeros into dhidden
// where a row is left out.  For the gradient alone also what it needs of a
// row: the target's logit is a dot product of the row with one of the weights.
// FUSED: the places, too.
template <typename E, bool FUSED>
__global__ void __launch_bounds__(256)
ce_rows_kernel(CeArgs a, int64_t dp, E *hc, E *hc2, int *count, int *row_of, const int *place, CeRow *rows, float *inv,
               float *loss, float *lse, bool zero_dh, bool grad_only, bool wide, bool wide_w, int *status) {
  constexpr int N = Vec16<E>::N;
  griddep_launch();
  griddep_wait();
  const int t = (int)(((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  int at, n;
  CeRow info = {0.f, 0.f, 0.f, -1};
  if (FUSED) {
    __shared__ uint32_t flags[CE_FUSE / 32];  // rows that count
    auto target = [&](int i) {
      return a.targets64 ? ((const int64_t *)a.targets)[i] : (int64_t)((const int32_t *)a.targets)[i];
    };
    constexpr int M = CE_FUSE / 256;
    int64_t id[M];  // all loads in flight
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int i = j * 256 + threadIdx.x;
      id[j] = i < a.T ? target(i) : a.ignore_index;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int i = j * 256 + threadIdx.x;
      const bool in = id[j] >= 0 && id[j] < a.V;
      if (!in && id[j] != a.ignore_index) record_status(status, STATUS_BAD_TARGET);
      const unsigned vote = __ballot_sync(FULL_MASK, in && id[j] != a.ignore_index && i < a.T);
      if (lane == 0) flags[i / 32] = vote;
    }
    __syncthreads();
    // Lane i has the four words of rows 128 i and on.
    int before = 0, all = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int w = lane * 4 + j;
      const uint32_t b = flags[w];
      all += __popc(b);
      if (w * 32 + 32 <= t) before += __popc(b);
      else if (w * 32 < t) before += __popc(b & ((1u << (t - w * 32)) - 1));
    }
    for (int d = 16; d; d >>= 1) {
      before += __shfl_xor_sync(FULL_MASK, before, d);
      all += __shfl_xor_sync(FULL_MASK, all, d);
    }
    n = all;
    at = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0) *count = n;
    if (t < a.T && (flags[t / 32] >> (t & 31) & 1)) {
      at = before;
      info.target = (int)target(t);
      if (lane == 0) row_of[at] = t;
    }
    if (t < a.T && at < 0 && lane == 0) {
      if (loss) loss[t] = 0.f;
      if (lse) lse[t] = 0.f;
    }
  } else {
    n = *count;
    at = t < a.T ? place[t] : -1;
    if (at >= 0) info = rows[at];
  }
  const E *src = nullptr;
  float f = 1.f;
  if (t < a.T) {
    if (at < 0) {
      if (zero_dh)
        for (int c = lane; c < a.D; c += 32) ((E *)a.dh)[t * a.ld_dh + c] = Elem<E>::from_f32(0.f);
      return;
    }
    src = (const E *)a.hidden + t * a.ld_h;
    if (grad_only) {
      const E *w = (const E *)a.weight + info.target * a.ld_w;
      float x = 0.f;
      if (wide && wide_w) {
        for (int u = lane; u < a.D / N; u += 32) {
          float p[N], q[N];
          Vec16<E>::load(src + u * N, p);
          Vec16<E>::load(w + u * N, q);
#pragma unroll
          for (int i = 0; i < N; ++i) x = fmaf(p[i], q[i], x);
        }
      } else {
        for (int c = lane; c < a.D; c += 32) x = fmaf(Elem<E>::load(src + c), Elem<E>::load(w + c), x);
      }
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(FULL_MASK, x, d);
      const float l = a.lse[t];
      f = grad_row<E>(info, a.scale * a.dloss[t], l, fmaf(-x, a.scale, l), a.z_loss);
      if (lane == 0) inv[at] = f;
    }
  } else {
    at = n + (t - a.T);
    if (at >= (int)round_up(n, CE_ROWS)) return;
  }
  if (lane == 0) rows[at] = info;
  put_row<E, false>(hc + at * dp, src, a.D, dp, 1.f, wide, lane);
  if (grad_only && sizeof(E) == 2) put_row<E, true>(hc2 + at * dp, src, a.D, dp, f, wide, lane);
}

// Weights whose rows do not start on 16-byte boundaries, copied to where they do.
__global__ void __launch_bounds__(256)
ce_weight_copy_kernel(int64_t V, int D, int64_t ld, int64_t ldw, const __nv_bfloat16 *w, __nv_bfloat16 *wc) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  for (int64_t v = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; v < V; v += (int64_t)gridDim.x * 8)
    for (int c = lane; c < (int)ldw; c += 32)
      wc[v * ldw + c] = c < D ? w[v * ld + c] : __float2bfloat16_rn(0.f);
}

// ------------------------------------------------------------- the rows' statistics
// A CTA joins 8 rows (64 bytes of each part): a row has 64 threads, which take
// every 64th part each, first the maximum of eight parts at a time, then
// their sums; the 64 results are joined in order of the threads.  The parts
// are without the target's logit x_t, which comes in last: with o the sum of the others'
// e^(x - x_t), lse - x_t = log(1 + o) keeps its bits where the model is
// nearly sure, and a sum that had a 1 in it would have lost o.  In a step
// also what the gradient needs of the rows, and the rows over their factors.
constexpr int JOIN_ROWS = 8, JOIN_THREADS = 512;
template <typename E>
__global__ void __launch_bounds__(JOIN_THREADS)
ce_join_kernel(const int *count, int nparts, int tpad, const float2 *part, const float *xt, const int *row_of,
               CeRow *rows, float *inv, float *loss, float *lse, const float *dloss, float scale, float z, const E *hc,
               E *hc2, int64_t dp) {
  griddep_launch();
  griddep_wait();
  constexpr int SL = JOIN_THREADS / JOIN_ROWS;
  __shared__ float2 sh[SL][JOIN_ROWS];
  __shared__ float factor[JOIN_ROWS];
  const int n = *count, r0 = blockIdx.x * JOIN_ROWS;
  if (r0 >= (dloss ? (int)round_up(n, CE_ROWS) : n)) return;
  const int sl = threadIdx.x / JOIN_ROWS, q = threadIdx.x % JOIN_ROWS;
  const float2 *p = part + r0 + q;
  float m = -INFINITY, s = 0.f;
  if (r0 < n) {
    for (int i = sl; i < nparts; i += 8 * SL) {
      float2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = i + j * SL;
        v[j] = k < nparts ? p[(int64_t)k * tpad] : make_float2(-INFINITY, 0.f);
      }
      float big = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) big = fmaxf(big, v[j].x);
      const float ref = big == -INFINITY ? 0.f : big;
      s *= exp2f(m - ref);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j].y * exp2f(v[j].x - ref);
      m = big;
    }
  }
  sh[sl][q] = make_float2(m, s);
  __syncthreads();
  // A warp's quarter of the 64 (rows across the lanes), then the four of a row.
  if (threadIdx.x < 32) {
    const int row = threadIdx.x & 7, part4 = threadIdx.x >> 3;
    m = -INFINITY;
    s = 0.f;
    auto add = [&](float2 o) {
      const float big = fmaxf(m, o.x), ref = big == -INFINITY ? 0.f : big;
      s = s * exp2f(m - ref) + o.y * exp2f(o.x - ref);
      m = big;
    };
#pragma unroll
    for (int i = 0; i < SL / 4; ++i) add(sh[part4 * (SL / 4) + i][row]);
    float2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i].x = __shfl_sync(FULL_MASK, m, row + 8 * i);
      o[i].y = __shfl_sync(FULL_MASK, s, row + 8 * i);
    }
    m = -INFINITY;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) add(o[i]);
    const int r = r0 + row;
    if (part4 == 0) {
      float f = 1.f;
      if (r < n) {
        const float x = xt[r];  // (in units of log 2, as m)
        float l, nll;
        if (m <= x) {
          nll = log1pf(s * exp2f(m - x));
          l = fmaf(x, LN2, nll);
        } else {  // the target's e^(x_t - m) beside the others' sum
          const float ln = logf(s) + log1pf(exp2f(x - m) / s);
          nll = fmaf(m - x, LN2, ln);
          l = fmaf(m, LN2, ln);
        }
        const int t = row_of[r];
        loss[t] = fmaf(z * l, l, nll);
        if (lse) lse[t] = l;
        if (dloss) {
          CeRow info = rows[r];
          f = grad_row<E>(info, scale * dloss[t], l, nll, z);
          rows[r] = info;
          inv[r] = f;
        }
      }
      factor[row] = f;
    }
  }
  if (!dloss || sizeof(E) != 2) return;
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp >= JOIN_ROWS) return;
  const int64_t at = (r0 + warp) * dp;
  put_row<E, true>(hc2 + at, hc + at, (int)dp, dp, factor[warp], true, threadIdx.x & 31);
}

// dhidden's sums of the chunks of one piece, in order, onto those of the pieces before.
template <typename E>
__global__ void __launch_bounds__(256)
ce_planes_kernel(const int *count, const int *row_of, const float *inv, int D, int64_t dp, int tpad, int nplanes, const float *planes,
                 float *acc, E *dh, int64_t ld_dh, bool first, bool last) {
  griddep_launch();
  griddep_wait();
  const int n = *count;
  const int64_t plane = (int64_t)tpad * dp;
  for (int64_t r = blockIdx.y; r < n; r += gridDim.y) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= D) continue;
    const int64_t at = r * dp + c;
    float4 s = first ? *(const float4 *)(planes + at) : *(const float4 *)(acc + at);
#pragma unroll 4
    for (int i = first ? 1 : 0; i < nplanes; ++i) {
      const float4 p = *(const float4 *)(planes + i * plane + at);
      s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
    }
    if (!last) {
      *(float4 *)(acc + at) = s;
      continue;
    }
    const float f = sizeof(E) == 2 ? inv[r] : 1.f;
    const float v[4] = {s.x * f, s.y * f, s.z * f, s.w * f};
    E *out = dh + row_of[r] * ld_dh + c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < D) out[j] = Elem<E>::from_f32(v[j]);
  }
}

// ------------------------------------------------------------- the call
size_t ce_scratch_bytes(const CeArgs &a, int mode) { return ce_layout(a, mode).bytes; }

template <typename E>
static cudaError_t run(const CeArgs &a, int mode, uint8_t *w, int *status, cudaStream_t stream) {
  const CeLayout l = ce_layout(a, mode);
  const bool grad = mode & CE_GRAD, loss = mode & CE_LOSS;
  int *count = (int *)(w + l.count), *row_of = (int *)(w + l.row_of), *place = (int *)(w + l.place);
  CeRow *rows = (CeRow *)(w + l.rows);
  E *hc = (E *)(w + l.hc), *hc2 = (E *)(w + l.hc2);
  float *inv = (float *)(w + l.inv);
  cudaError_t e;
  float *lo = loss ? a.loss : nullptr, *ls = loss ? a.lse : nullptr;
  const bool fused = a.T <= CE_FUSE;
  if (!fused) {
    if (a.targets64)
      e = launch_pdl(ce_places_kernel<int64_t>, dim3(1), dim3(1024), 0, stream, a.T, a.V, a.ignore_index,
                     (const int64_t *)a.targets, count, row_of, place, rows, lo, ls, status);
    else
      e = launch_pdl(ce_places_kernel<int32_t>, dim3(1), dim3(1024), 0, stream, a.T, a.V, a.ignore_index,
                     (const int32_t *)a.targets, count, row_of, place, rows, lo, ls, status);
    if (e != cudaSuccess) return e;
  }
  constexpr int N = Vec16<E>::N;
  const bool wide = a.D % N == 0 && a.ld_h % N == 0 && ((uintptr_t)a.hidden & 15) == 0;
  const bool wide_w = a.ld_w % N == 0 && ((uintptr_t)a.weight & 15) == 0;
  e = launch_pdl(fused ? ce_rows_kernel<E, true> : ce_rows_kernel<E, false>,
                 dim3((unsigned)ceil_div((int64_t)a.T + CE_ROWS, 8)), dim3(256), 0, stream, a, l.dp, hc, hc2, count, row_of,
                 (const int *)place, rows, inv, lo, ls, grad, grad && !loss, wide, wide_w, status);
  if (e != cudaSuccess) return e;
  if (l.ldw) {
    e = launch_pdl(ce_weight_copy_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(a.V, 8), 8 * 152)), dim3(256), 0,
                   stream, (int64_t)a.V, a.D, a.ld_w, l.ldw, (const __nv_bfloat16 *)a.weight, (__nv_bfloat16 *)(w + l.wc));
    if (e != cudaSuccess) return e;
  }
  CeMats m = {};
  m.V = a.V;
  m.D = a.D;
  m.tpad = l.tpad;
  m.ldh = l.dp;
  m.ldw = l.ldw ? l.ldw : a.ld_w;
  m.ldg = l.ldg;
  m.count = count;
  m.row_of = row_of;
  m.rows = rows;
  m.inv = inv;
  m.h = hc;
  m.h2 = hc2;
  m.w = l.ldw ? w + l.wc : a.weight;
  m.g = w + l.g;
  m.scale = a.scale;
  m.part = (float2 *)(w + l.part);
  m.xt = (float *)(w + l.xt);
  m.gf32 = a.gf32;
  m.accumulate = a.accumulate;
  m.dh = a.dh;
  m.dw = a.dw;
  m.ld_dh = a.ld_dh;
  m.planes = (float *)(w + l.acc);
  m.acc = m.planes + (l.per_piece > 1 ? (int64_t)l.per_piece * l.tpad * l.dp : 0);
  m.status = status;
  if (loss) {
    if ((e = a.f32 ? ce_simt_stats(m, stream) : ce_tc_stats(m, stream)) != cudaSuccess) return e;
    e = launch_pdl(ce_join_kernel<E>, dim3(l.tpad / JOIN_ROWS), dim3(JOIN_THREADS), 0, stream, (const int *)count, l.nparts, l.tpad,
                   (const float2 *)m.part, (const float *)m.xt, (const int *)row_of, rows, inv, a.loss, a.lse,
                   (const float *)(grad ? a.dloss : nullptr), a.scale, a.z_loss, (const E *)hc, hc2, l.dp);
    if (e != cudaSuccess) return e;
  }
  if (!grad) return cudaSuccess;
  for (int i = 0; i < l.npieces; ++i) {
    CePiece p = {};
    p.chunk = l.chunk;
    p.v0 = i * l.per_piece * l.chunk;
    p.n = std::min(l.per_piece * l.chunk, a.V - p.v0);
    p.nchunks = (int)ceil_div(p.n, l.chunk);
    p.first = i == 0;
    p.last = i + 1 == l.npieces;
    CeMats mp = m;
    if (l.per_piece == 1) mp.planes = nullptr;
    if ((e = a.f32 ? ce_simt_logits_grad(mp, p, stream) : ce_tc_logits_grad(mp, p, stream)) != cudaSuccess) return e;
    if ((e = a.f32 ? ce_simt_grads(mp, p, stream) : ce_tc_grads(mp, p, stream)) != cudaSuccess) return e;
    if (l.per_piece > 1) {
      e = launch_pdl(ce_planes_kernel<E>, dim3((unsigned)ceil_div(a.D, 1024), (unsigned)std::min(l.tpad, 16384)), dim3(256),
                     0, stream, (const int *)count, (const int *)row_of, (const float *)m.inv, a.D, l.dp, l.tpad, p.nchunks,
                     (const float *)mp.planes, mp.acc, (E *)a.dh, a.ld_dh, p.first, p.last);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

// dweight where there are no rows at all.
__global__ void __launch_bounds__(256) ce_zero_kernel(int64_t bytes2, uint16_t *p) {
  griddep_launch();
  griddep_wait();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < bytes2; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

cudaError_t launch_linear_ce(const CeArgs &a, int mode, void *scratch, int *status, cudaStream_t stream) {
  if (a.T == 0) {
    if (!(mode & CE_GRAD) || a.accumulate) return cudaSuccess;
    return launch_pdl(ce_zero_kernel, dim3(1216), dim3(256), 0, stream, (int64_t)a.V * a.D * (a.gf32 ? 2 : 1),
                      (uint16_t *)a.dw);
  }
  return a.f32 ? run<float>(a, mode, (uint8_t *)scratch, status, stream)
               : run<__nv_bfloat16>(a, mode, (uint8_t *)scratch, status, stream);
}

}  // namespace moe

// The linear cross entropy's matrix products in float, on CUDA cores.
//
// Products of floats need 24 bits, which the tensor cores' formats do not
// hold, so float models (small ones, and checks) take FFMA: tiles of 128 x
// 128 outputs (64 x 64 where those would leave SMs without one), 256 threads
// with 8 x 8 (4 x 4) outputs each, K steps of 16 through shared memory, one
// step ahead in registers.  The epilogues are those of the
// tensor-core kernels: the same statistics per 64 columns, the same pieces.
// Each output is summed over K in order.
//
// Bound by FFMA and by shared memory's reads (four of 16 bytes for 64 FMAs):
// a step of 1024 x 512 x 16000 takes 1273 us, 53 TFLOP/s over its four
// products.  Small ones wait for their loads: 147 us at 333 x 256 x 5003 (tiles of
// 64 threads with 8 x 8 outputs each, which read shared memory less, took 271).
#include "linear_ce.h"
#include "tc_host.h"

namespace moe {

constexpr int SM_STATS = 0, SM_LOGITS = 1, SM_DH = 2, SM_DW = 3;
constexpr int SK = 16;

struct SimtParams {
  CeMats m;
  CePiece p;
  int nparts;
};

// Four consecutive floats of a matrix, those past `n` as zeros.
__device__ inline float4 four(const float *p, int n, bool wide) {
  if (n >= 4 && wide) return *(const float4 *)p;
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}

// An operand of one tile: 64 S rows (of the output's rows or columns) x 16 K,
// S units of four floats a thread.  KMAJOR: K runs along the row.
template <bool KMAJOR, int S>
struct Operand {
  const float *p;
  int64_t ld;
  int rows, k;  // valid extents from the tile's origin
  bool wide;    // units are on 16-byte boundaries
  float4 r[S];
  __device__ void load(int k0) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int u = threadIdx.x + 256 * i;
      if (KMAJOR) {
        const int row = u >> 2, kk = k0 + (u & 3) * 4;
        r[i] = row < rows ? four(p + row * ld + kk, k - kk, wide) : make_float4(0, 0, 0, 0);
      } else {
        const int kk = k0 + u / (16 * S), row = u % (16 * S) * 4;
        r[i] = kk < k ? four(p + kk * ld + row, rows - row, wide) : make_float4(0, 0, 0, 0);
      }
    }
  }
  __device__ void store(float (*s)[64 * S + 4]) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int u = threadIdx.x + 256 * i;
      if (KMAJOR) {
        const int row = u >> 2, kk = (u & 3) * 4;
        s[kk][row] = r[i].x;
        s[kk + 1][row] = r[i].y;
        s[kk + 2][row] = r[i].z;
        s[kk + 3][row] = r[i].w;
      } else {
        *(float4 *)&s[u / (16 * S)][u % (16 * S) * 4] = r[i];
      }
    }
  }
};

// Tile (bx, by) of a product, for dhidden of chunk bz.  sA, sB: two buffers each.
template <int KIND, int S>
__device__ inline void simt_tile(const SimtParams &a, float (*sA)[SK][64 * S + 4], float (*sB)[SK][64 * S + 4], int bx,
                                 int by, int bz) {
  const CeMats &m = a.m;
  const CePiece &pc = a.p;
  constexpr int ST = 64 * S, RT = 4 * S;
  const int count = *m.count;
  const int r0 = bx * ST, c0 = by * ST;  // the tile's rows and columns
  if (KIND != SM_DW && r0 >= (KIND == SM_LOGITS ? (int)round_up(count, CE_ROWS) : count)) return;
  const float *h = (const float *)m.h, *w = (const float *)m.w, *g = (const float *)m.g;
  const bool ww = m.ldw % 4 == 0 && ((uintptr_t)m.w & 15) == 0;
  constexpr bool AK = KIND != SM_DW, BK = KIND == SM_STATS || KIND == SM_LOGITS;
  Operand<AK, S> A;
  Operand<BK, S> B;
  A.wide = true;
  const int v0 = pc.v0;
  int k;
  if (KIND == SM_STATS || KIND == SM_LOGITS) {
    k = m.D;
    A.p = h + r0 * m.ldh; A.ld = m.ldh; A.rows = m.tpad - r0;
    B.p = w + (v0 + c0) * m.ldw; B.ld = m.ldw; B.rows = m.V - v0 - c0; B.wide = ww;
  } else if (KIND == SM_DH) {
    const int ch = bz * pc.chunk;
    k = min(pc.chunk, pc.n - ch);
    A.p = g + r0 * m.ldg + ch; A.ld = m.ldg; A.rows = m.tpad - r0;
    B.p = w + (v0 + ch) * m.ldw + c0; B.ld = m.ldw; B.rows = m.D - c0; B.wide = ww;
  } else {
    k = count;
    A.p = g + r0; A.ld = m.ldg; A.rows = pc.n - r0;
    B.p = h + c0; B.ld = m.ldh; B.rows = m.D - c0; B.wide = true;
  }
  A.k = B.k = k;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  // A thread's rows are r0 + 4 ty + {0..3} and + 64, its columns alike.
  F2 sum[RT][RT / 2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < RT / 2; ++j) sum[i][j] = F2(0.f);
  A.load(0);
  B.load(0);
  int buf = 0;
  for (int k0 = 0; k0 < k; k0 += SK) {
    A.store(sA[buf]);
    B.store(sB[buf]);
    __syncthreads();
    if (k0 + SK < k) {
      A.load(k0 + SK);
      B.load(k0 + SK);
    }
#pragma unroll
    for (int kk = 0; kk < SK; ++kk) {
      float4 x[S], y[S];
#pragma unroll
      for (int h = 0; h < S; ++h) {
        x[h] = *(const float4 *)&sA[buf][kk][64 * h + ty * 4];
        y[h] = *(const float4 *)&sB[buf][kk][64 * h + tx * 4];
      }
#pragma unroll
      for (int h = 0; h < S; ++h) {
        const F2 y0(y[h].x, y[h].y), y1(y[h].z, y[h].w);
#pragma unroll
        for (int g = 0; g < S; ++g) {
          const float v[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 d(v[i]);
            sum[4 * g + i][2 * h] = fma2(d, y0, sum[4 * g + i][2 * h]);
            sum[4 * g + i][2 * h + 1] = fma2(d, y1, sum[4 * g + i][2 * h + 1]);
          }
        }
      }
    }
    buf ^= 1;  // the other buffer was last read before the barrier of this step
  }
  float acc[RT][RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < RT / 2; ++j) sum[i][j].get(acc[i][2 * j], acc[i][2 * j + 1]);
  auto rowof = [&](int i) { return (i & 3) + (i >> 2) * 64 + ty * 4; };
  auto colof = [&](int j) { return (j & 3) + (j >> 2) * 64 + tx * 4; };
  constexpr float L2E = 1.44269504088896340736f;
  if (KIND == SM_STATS) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = r0 + rowof(i);
      const int target = m.rows[row].target - c0;
#pragma unroll
      for (int hf = 0; hf < S; ++hf) {  // 64 columns each
        float big = -INFINITY, s = 0.f;
#pragma unroll
        for (int j = 4 * hf; j < 4 * hf + 4; ++j) {
          const int c = colof(j);
          const float x = acc[i][j] * (m.scale * L2E);
          if (c == target) m.xt[row] = x;
          acc[i][j] = c0 + c < m.V && c != target ? x : -INFINITY;
          big = fmaxf(big, acc[i][j]);
        }
        for (int d = 8; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(FULL_MASK, big, d));
        const float ref = big == -INFINITY ? 0.f : big;
#pragma unroll
        for (int j = 4 * hf; j < 4 * hf + 4; ++j) s += exp2f(acc[i][j] - ref);
        for (int d = 8; d; d >>= 1) s += __shfl_xor_sync(FULL_MASK, s, d);
        const int part = by * S + hf;
        if (tx == 0 && part < a.nparts) m.part[(int64_t)part * m.tpad + row] = make_float2(big, s);
      }
    }
  } else if (KIND == SM_LOGITS) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = r0 + rowof(i);
      const CeRow R = m.rows[row];
      const int target = R.target - v0 - c0;
      const bool zero = R.c == 0.f && R.b == 0.f;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int c = colof(j);
        float x = R.c * exp2f(fmaf(acc[i][j], m.scale * L2E, -R.lse2));
        if (c == target) x = R.b;
        acc[i][j] = zero || v0 + c0 + c >= m.V ? 0.f : x;
      }
      float *out = (float *)m.g + row * m.ldg + c0 + tx * 4;
#pragma unroll
      for (int h = 0; h < S; ++h)
        *(float4 *)(out + 64 * h) = make_float4(acc[i][4 * h], acc[i][4 * h + 1], acc[i][4 * h + 2], acc[i][4 * h + 3]);
    }
  } else if (KIND == SM_DH) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = r0 + rowof(i);
      if (row >= count) continue;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int c = c0 + colof(j);
        if (c >= m.D) continue;
        const int64_t at = row * m.ldh + c;
        if (m.planes) {
          m.planes[(int64_t)bz * m.tpad * m.ldh + at] = acc[i][j];
          continue;
        }
        const float x = pc.first ? acc[i][j] : m.acc[at] + acc[i][j];
        if (pc.last) ((float *)m.dh)[m.row_of[row] * m.ld_dh + c] = x;
        else m.acc[at] = x;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = r0 + rowof(i);
      if (row >= pc.n) continue;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int c = c0 + colof(j);
        if (c >= m.D) continue;
        float *o = (float *)m.dw + (int64_t)(v0 + row) * m.D + c;
        *o = m.accumulate ? *o + acc[i][j] : acc[i][j];
      }
    }
  }
}

// The logits' products: a grid of tiles.
template <int KIND, int S>
__global__ void __launch_bounds__(256, S == 2 ? 2 : 4) ce_simt_kernel(const SimtParams a) {
  griddep_launch();
  griddep_wait();
  __shared__ float sA[2][SK][64 * S + 4], sB[2][SK][64 * S + 4];
  simt_tile<KIND, S>(a, sA, sB, blockIdx.x, blockIdx.y, 0);
}

// Both products of g, side by side in one launch (they have little more than a
// wave of tiles each at the sizes that float models have): dhidden's tiles,
// rows fastest, then dweight's.
template <int S>
__global__ void __launch_bounds__(256, S == 2 ? 2 : 4) ce_simt_grads_kernel(const SimtParams a, int mt, int nt, int ndh, int vt) {
  griddep_launch();
  griddep_wait();
  __shared__ float sA[2][SK][64 * S + 4], sB[2][SK][64 * S + 4];
  const int i = blockIdx.x;
  if (i < ndh) simt_tile<SM_DH, S>(a, sA, sB, i % mt, i / mt % nt, i / mt / nt);
  else simt_tile<SM_DW, S>(a, sA, sB, (i - ndh) % vt, (i - ndh) / vt, 0);
}

// Whether tiles of 128 x 128 fill the SMs twice.
static bool large(int64_t tiles) { return tiles >= 2 * device_sms(); }

template <int KIND>
static cudaError_t launch(const CeMats &m, const CePiece &p, int64_t rows, int64_t cols, cudaStream_t stream) {
  SimtParams a = {m, p, (int)ceil_div(m.V, CE_PART)};
  auto grid = [&](int t) { return dim3((unsigned)ceil_div(rows, t), (unsigned)ceil_div(cols, t)); };
  if (large(ceil_div(rows, 128) * ceil_div(cols, 128)))
    return launch_pdl(ce_simt_kernel<KIND, 2>, grid(128), dim3(256), 0, stream, a);
  return launch_pdl(ce_simt_kernel<KIND, 1>, grid(64), dim3(256), 0, stream, a);
}

cudaError_t ce_simt_stats(const CeMats &m, cudaStream_t stream) {
  CePiece p = {};
  p.n = m.V;
  return launch<SM_STATS>(m, p, m.tpad, m.V, stream);
}

cudaError_t ce_simt_logits_grad(const CeMats &m, const CePiece &p, cudaStream_t stream) {
  return launch<SM_LOGITS>(m, p, m.tpad, p.n, stream);
}

cudaError_t ce_simt_grads(const CeMats &m, const CePiece &p, cudaStream_t stream) {
  SimtParams a = {m, p, (int)ceil_div(m.V, CE_PART)};
  auto tiles = [&](int t, int &mt, int &nt, int &ndh, int &vt) {
    mt = (int)ceil_div(m.tpad, t);
    nt = (int)ceil_div(m.D, t);
    ndh = mt * nt * p.nchunks;
    vt = (int)ceil_div(p.n, t);
    return (unsigned)(ndh + vt * nt);
  };
  int mt, nt, ndh, vt;
  unsigned n = tiles(128, mt, nt, ndh, vt);
  if (large(n)) return launch_pdl(ce_simt_grads_kernel<2>, dim3(n), dim3(256), 0, stream, a, mt, nt, ndh, vt);
  n = tiles(64, mt, nt, ndh, vt);
  return launch_pdl(ce_simt_grads_kernel<1>, dim3(n), dim3(256), 0, stream, a, mt, nt, ndh, vt);
}

}  // namespace moe

// Matrix products of the linear cross entropy on CTA pairs (tcgen05, bf16).
//
// Three persistent kernels on one skeleton; an item is a tile of 256 x 256
// outputs of one product, run by a cluster of two CTAs as M = 256 MMAs
// (cta_group::2): each CTA holds 128 rows of A and half of B's columns, and
// its tensor memory receives 128 rows of the tile.
//
//   STATS   x[t, v] = sum_d h[t, d] w[v, d]     epilogue: for each row and 64 columns the
//           maximum and the sum of exponentials of all but the target, and the target's logit
//   LOGITS  the same product for the columns of a piece; epilogue: g, one
//           rounding to bf16, by TMA stores
//   GRADS   dh[t, d] = sum_v g[t, v] w[v, d]    (A K-major, B MN-major)
//           dw[v, d] = sum_t g[t, v] h2[t, d]   (both MN-major; h2: h over the row's factor)
//           in one launch: the two have the same tiles and, at 8192 rows,
//           the same K, so that together they fill the last wave better
//
// Rows of the accumulator are tokens in the first two, so a thread of the
// epilogue has a row's columns in its own lane and takes maximum and sum
// without a shuffle.  Two accumulators of 256 columns alternate: an item's
// epilogue runs under the next item's MMAs.  A stage is two K blocks of 64: 32
// KB of A and 32 KB of B a CTA, three of them; where a few rows are all there
// is, a stage has room for those alone (the MMAs read on into B's bytes for
// rows that nobody looks at) and there are five: reading the weights is bound
// by the bytes in flight then (5 rows x 2048 x 32000: 33.1 us with three, 31.3
// with five).  Every output is summed in K blocks of 64 in order; the tile it
// falls in does not change that.
//
// What bounds them: the tensor cores.  A forward of 4096 x 2048 x 50257 takes 433
// us in a burst (1.95 PFLOP/s; a large cuBLAS product: 1.90) and 487 in a long
// run under the power cap (1.73; 1.71); a step of 8192 x 2048 x 131072 10.6 ms, 1.66
// PFLOP/s over its four products.  Counters at 4096 x 2048 x 24576: the tensor pipe
// is busy 89 % of STATS, 79 % of LOGITS, 84 % of GRADS.  At few columns of K (1000) the SMs' reads of L2 (64 KB a K block and
// pair, 13 TB/s in all) share it with g's stores, and LOGITS takes a fifth longer than its MMAs.
#include <cuda.h>

#include "linear_ce.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

using namespace umma;

constexpr int CE_STATS = 0, CE_LOGITS = 1, CE_GRADS = 2;
constexpr int CT_TILE = 16384;  // a K block of 64: 128 rows of A, or half of B's columns, of a CTA
// Epilogue warps: eight for the gradients, half of the columns each, with a
// staging tile of 4 KB; for the logits sixteen with a quarter each, so that a
// thread's sums over the K chunks (64) stay in registers (and 2 KB each for g:
// 16-byte stores past shared memory made a step of 8192 x 2048 x 131072 11.0 ms,
// 32-byte ones 10.75, these 10.6).  Stages of two K blocks: one handshake
// and one commit for eight MMAs (forward 4096 x 2048 x 50257: 527 us with one block,
// 459 with two; the gradients' products 1620 and 1569; three blocks leave too
// few stages: 1720).
constexpr int CT_EPI_FIRST = 4, SUB = 2;
template <int KIND>
struct CtCfg {
  static constexpr int EPI_WARPS = KIND == CE_GRADS ? 8 : 16;
  static constexpr int THREADS = 32 * (CT_EPI_FIRST + EPI_WARPS);
  static constexpr int STG_WARP = KIND == CE_STATS ? 0 : KIND == CE_LOGITS ? 2048 : 4096;  // staging tile of a warp
  static constexpr int STG_BYTES = EPI_WARPS * STG_WARP;
  static constexpr int RING = 7 * 2 * CT_TILE - STG_BYTES;  // bytes of the stages
  static constexpr int SMEM = 1024 + RING + STG_BYTES + 512;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};
constexpr int CT_PREFETCH = 8;  // K blocks (none: 33.3 us at 5 rows x 2048 x 32000, 8 or 16: 31.3, 32: 35.5)
constexpr int CT_MAX_STAGES = 5;
constexpr uint32_t CT_HINT = 100000;  // ns
constexpr uint32_t CT_TMEM_COLS = 512;
// The logits are summed in chunks of 512 of K, each in an
// accumulator of its own, and the chunks in FP32 registers: the tensor cores
// cut each of their sums off instead of rounding it, which leaves a loss
// 1.0e-6 off at K = 2048 in one chain, 5e-7 in chunks of 1024 and 2.4e-7 in
// chunks of 512 (1.1e-7 in 256; a rounded FP32 product of the kind that keeps
// its logits: 4.6e-7).  512 takes 2 to 3 % more time than 1024, 256 six more.
// The gradient's logits are summed the same way and have the same bits, so that
// probabilities add up to 1 however far the sums are off: in one chain a row of
// 16384 addends that make 60 was short by 4.2e-3 of that (a step of 8192 x 2048 x
// 131072 takes 10.6 ms for 10.4 with one).
constexpr int CT_KCHUNK = 8;   // a multiple of SUB
// An accumulator of the gradients' products takes no more than this of a sum, in K
// blocks (of dweight 8192 rows, as many as a chunk of dhidden has columns).  What
// is left of a longer one goes into the other accumulator, and the epilogue
// adds the sum so far onto it in FP32, rounded: the tensor cores cut off what
// an addend has below 2^-23 of the sum, always towards zero (2^21 rows of one
// sign in one chain: 1.1e-2 of dweight lost, in chains of 8192: 5e-7).
template <int KIND>
constexpr int CT_CHAIN = KIND == CE_GRADS ? 128 : CT_KCHUNK;
constexpr float CE_LOG2E = 1.44269504088896340736f;

struct CtMaps {
  CUtensorMap h, w, g;     // K-major tiles: boxes of 128 rows x 64
  CUtensorMap h32, w32;    // the same rows, 32 at a time
  CUtensorMap ht, wt, gt;  // MN-major tiles: boxes of 64 rows x 64, two blocks of columns at once
  CUtensorMap ht1, wt1;    // one block of columns
  CUtensorMap gout;        // 32 rows x 32: g's stores
  CUtensorMap dw;          // dweight: 32 rows x 128 bytes
};

struct CtParams {
  int V, D, tpad;
  const int *count;
  const int *row_of;
  const CeRow *rows;
  const float *inv;
  float s2;  // scale * log2(e)
  float2 *part;
  float *xt;
  int v0, n, chunk, nchunks;  // the piece
  bool first, last;
  bool w_blocks, dw_tma, accumulate, gf32, dh_wide;
  __nv_bfloat16 *dh;
  int64_t ld_dh, ldh;
  void *dw;
  float *acc, *planes;
  int *status;
};

struct CtItem {
  int kind;   // 0: logits, 1: dhidden, 2: dweight
  int m, chunk, nk;
  int n0;     // first column of the tile: of the piece's vocabulary (logits), of D (gradients)
  int cols;   // columns of the tile: a multiple of 64 up to 256 (gradients: 128 or 256)
};

// The items of a pair, in order.
//
// Logits, one row tile (few rows, bound by reading the weights): the
// vocabulary in units of 64 columns, a contiguous run of them to each pair, so
// that no pair has more than one unit above the mean (32000 x 2048: 7 units
// instead of two whole tiles of 4).  More row tiles: tiles of 256 columns, row
// tiles fastest, so that a tile of the weights is read by all of them at about
// the same time; narrower ones where a wave of whole tiles would be empty for the most part.
//
// Gradients: the items of the product with the longer sums (dhidden's up to
// 8192 rows, dweight's above) are dealt out in turn; the pairs that have one
// less of them get as many more of the other's as make up for it, the rest goes round.
template <int KIND>
struct CtWork {
  int count, mt, kd, kr;
  int it, end;                   // logits: the pair's next unit or tile, and the last one's end
  int nt, cols;
  int nl, ns, heavy, extra, delta, pair, pairs;  // gradients: longer items, shorter ones
  bool long_dw;
  bool run;
  __device__ CtWork(const CtParams &p, int pair_, int pairs_) {
    pair = pair_;
    pairs = pairs_;
    // Not through the read-only path, whose loads may be moved above the wait
    // for the kernel that writes it.
    count = __shfl_sync(FULL_MASK, *(const volatile int *)p.count, 0);
    mt = (count + CE_ROWS - 1) / CE_ROWS;
    kd = (p.D + 63) / 64;
    kr = (count + 63) / 64;
    if (KIND == CE_GRADS) {
      nt = (p.D + 255) / 256;
      const int ndh = p.nchunks * mt * nt, ndw = (p.n + 255) / 256 * nt;
      // K blocks of an item; one of dweight takes the time of its stores (about five blocks) at least
      // (gradient of 256 x 2048 x 32000: 112.7 us when counted as eight, 106.7 as five, 118.7 as fourteen).
      const int kh = (min(p.chunk, p.n) + 63) / 64, kw = max(kr, 5);
      long_dw = kw > kh;
      nl = long_dw ? ndw : ndh;
      ns = long_dw ? ndh : ndw;
      heavy = nl % pairs;  // pairs with one more of the longer items
      const int kl = long_dw ? kw : kh, ks = long_dw ? kh : kw;
      delta = heavy ? (kl + ks / 2) / ks : 0;
      extra = min(ns, (pairs - heavy) * delta);
      it = 0;
      return;
    }
    run = mt == 1;
    if (run) {
      const int units = (p.n + 63) / 64;
      it = (int)((int64_t)units * pair / pairs);
      end = (int)((int64_t)units * (pair + 1) / pairs);
      return;
    }
    cols = 256;
    int best = 0x7fffffff;
    for (int c = 256; c >= 64; c -= 64) {  // waves x (columns + the cost of a tile by itself)
      const int waves = (mt * ((p.n + c - 1) / c) + pairs - 1) / pairs;
      if (waves * (c + 64) < best) {
        best = waves * (c + 64);
        cols = c;
      }
      if (waves > 8) break;  // (then the last wave does not matter)
    }
    nt = (p.n + cols - 1) / cols;
    it = pair;
    end = mt * nt;
  }
  __device__ bool next(const CtParams &p, CtItem &r) {
    r.chunk = 0;
    r.kind = 0;
    if (KIND != CE_GRADS) {
      if (it >= end) return false;
      r.nk = kd;
      if (run) {
        const int u = min(4, end - it);
        r.m = 0;
        r.n0 = it * 64;
        r.cols = u * 64;
        it += u;
      } else {
        r.m = it % mt;
        r.n0 = it / mt * cols;
        r.cols = cols;
        it += pairs;
      }
      return true;
    }
    const int own = nl / pairs + (pair < heavy ? 1 : 0);
    int i = it++;
    bool longer = i < own;
    if (longer) {
      i = pair + i * pairs;
    } else {
      i -= own;
      if (pair >= heavy && i < delta) {
        i = pair - heavy + i * (pairs - heavy);
        if (i >= extra) return false;  // (then there are no others)
      } else {
        i = extra + pair + (i - (pair >= heavy ? delta : 0)) * pairs;
        if (i >= ns) return false;
      }
    }
    r.kind = longer == long_dw ? 2 : 1;
    r.n0 = i % nt * 256;
    const int rest = i / nt;
    r.cols = p.D - r.n0 <= 128 ? 128 : 256;
    if (r.kind == 2) {
      r.m = rest;
      r.nk = kr;
    } else {
      r.m = rest % mt;
      r.chunk = rest / mt;
      r.nk = (min(p.chunk, p.n - r.chunk * p.chunk) + 63) / 64;
    }
    return true;
  }
};

// mbar_wait of these kernels: the thread is suspended for up to `hint` ns at a
// time instead of asking again and again.
__device__ inline bool ct_try_wait(uint64_t *bar, uint32_t parity, uint32_t hint) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint)
      : "memory");
  return ok != 0;
}
__device__ inline bool ct_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status) {
  if (ct_try_wait(bar, parity, CT_HINT)) return true;
  const uint64_t t0 = globaltimer();
  while (!ct_try_wait(bar, parity, CT_HINT)) {
    if (*abort_flag) return false;
    if (globaltimer() - t0 > WAIT_TIMEOUT_NS) {
      *abort_flag = 1;
      record_status(status, STATUS_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same by a whole warp, with one answer for all of it.
__device__ inline bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status) {
  return __all_sync(FULL_MASK, ct_wait(bar, parity, abort_flag, status));
}
// One lane of a whole warp, the same each time.
__device__ inline bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ inline float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Boxes of several blocks of 64 columns, for the pair's barrier.
__device__ inline void tma_load_3d_pair(void *dst, const CUtensorMap *m, uint32_t bar_cluster, int c0, int c1, int c2,
                                        uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster), "l"(policy)
      : "memory");
}
// A tile store with an L2 policy.
__device__ inline void tma_store_2d_hint(const CUtensorMap *m, const void *src, int c0, int c1, uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], %4;" ::"l"(m),
               "r"(c0), "r"(c1), "r"(smem_u32(src)), "l"(policy)
               : "memory");
}
// A tile on its way into L2.
__device__ inline void tma_prefetch_2d(const CUtensorMap *m, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(m), "r"(c0), "r"(c1) : "memory");
}
// A tile of 32 rows x 128 bytes from shared memory, added to what is there.
__device__ inline void tma_reduce_add_2d(const CUtensorMap *m, const void *src, int c0, int c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}

// ---- epilogues: a warp's 32 rows (lane = row) x half of the tile's columns ----
// v: the thread's 64 logits (columns from 64 cq of the tile), summed over the
// K chunks.
__device__ inline void stats_epilogue(const CtParams &p, const CtItem &im, float (&v)[64], int row, int cq) {
  const int col0 = im.n0 + cq * 64;
  const int target = p.rows[row].target - col0, left = p.V - col0;
  if (cq * 64 >= im.cols || left <= 0) return;
#pragma unroll
  for (int j = 0; j < 64; ++j) v[j] *= p.s2;
  if ((unsigned)target < 64u) {
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      x = target == j ? v[j] : x;
      v[j] = target == j ? -INFINITY : v[j];
    }
    p.xt[row] = x;
  }
  if (left < 64) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (j >= left) v[j] = -INFINITY;
  }
  float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int j = 4; j < 64; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
  float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const float ref = m == -INFINITY ? 0.f : m;  // (NaN does not get past fmaxf, but does get into the sum)
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 64; ++j) s[j & 3] += ex2(v[j] - ref);
  p.part[(int64_t)(col0 / 64) * p.tpad + row] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
}

// g of the same 64 columns from the same sums, 32 at a time through the
// warp's buffer: rows of 64 bytes, the 16-byte units of two rows together
// changed round as the 64-byte swizzle has them.
__device__ inline void logits_epilogue(const CtMaps &maps, const CtParams &p, const CtItem &im, const float (&v)[64],
                                       int row, int cq, uint8_t *stg, int lane) {
  const int pc = im.n0 + cq * 64;  // column in the piece
  if (cq * 64 >= im.cols || pc >= p.n) return;
  const CeRow R = p.rows[row];
  const bool zero = R.c == 0.f && R.b == 0.f;
  const int target = R.target - p.v0 - pc, left = p.V - p.v0 - pc;
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    if (lane == 0) bulk_wait_read<0>();  // the last store has read the buffer
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = c + 8 * u + 2 * i + k;
          x[k] = R.c * ex2(fmaf(v[j], p.s2, -R.lse2));
          if (j == target) x[k] = R.b;
          if (zero || j >= left) x[k] = 0.f;
        }
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[0], x[1]);
        w[i] = *(const uint32_t *)&b;
      }
      *(uint4 *)(stg + lane * 64 + ((u ^ (lane >> 1 & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&maps.gout, stg, pc + c, row);
      bulk_commit();
    }
  }
}

// 32 rows x 32 float columns of a warp through its buffer: f(row of the 32,
// column of the 32, four values) with eight lanes a row.
template <typename F>
__device__ inline void by_rows(uint8_t *stg, const float (&v)[32], int lane, F &&f) {
  if (lane == 0) bulk_wait_read<0>();  // a store of the item before has read the buffer
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *(float4 *)(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (lane >> 3) + 4 * i, ch = lane & 7;
    f(r, ch * 4, *(const float4 *)(stg + r * 128 + ((ch ^ (r & 7)) << 4)));
  }
  __syncwarp();
}

__device__ inline void dhidden_epilogue(const CtParams &p, const CtItem &im, uint32_t taddr, int row0, int count, int half,
                                        uint8_t *stg, int lane) {
  const int wcols = im.cols / 2, col0 = im.n0 + half * wcols;
  float *plane = p.planes ? p.planes + (int64_t)im.chunk * p.tpad * p.ldh : nullptr;
  for (int c = 0; c < wcols && col0 + c < p.D; c += 32) {
    float v[32];
    tmem_ld32(taddr + c, v);
    by_rows(stg, v, lane, [&](int r, int cc, float4 x) {
      const int row = row0 + r, col = col0 + c + cc;
      if (row >= count || col >= p.D) return;
      const int64_t at = row * p.ldh + col;
      if (plane) {
        *(float4 *)(plane + at) = x;
        return;
      }
      if (!p.first) {
        const float4 y = *(const float4 *)(p.acc + at);
        x.x = y.x + x.x; x.y = y.y + x.y; x.z = y.z + x.z; x.w = y.w + x.w;
      }
      if (!p.last) {
        *(float4 *)(p.acc + at) = x;
        return;
      }
      __nv_bfloat16 *out = p.dh + p.row_of[row] * p.ld_dh + col;
      const float f = p.inv[row];
      x.x *= f; x.y *= f; x.z *= f; x.w *= f;
      const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
      if (p.dh_wide) {
        *(uint2 *)out = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
      } else {
        const __nv_bfloat16 e[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < p.D) out[j] = e[j];
      }
    });
  }
}

// Where no row counts there is no accumulator, and the values are zero.
__device__ inline void dweight_epilogue(const CtMaps &maps, const CtParams &p, const CtItem &im, uint32_t taddr, int row0,
                                        int half, uint8_t *stg, int lane, uint64_t out_policy) {
  const int wcols = im.cols / 2, col0 = im.n0 + half * wcols;  // row0: row of dweight
  if (row0 >= p.V) return;
  for (int c = 0; c < wcols && col0 + c < p.D; c += p.gf32 || !p.dw_tma ? 32 : 64) {
    float v[2][32];
    if (im.nk == 0) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[0][j] = v[1][j] = 0.f;
    } else if (p.gf32 || !p.dw_tma) {
      tmem_ld32(taddr + c, v[0]);
    } else {
      tmem_ld32x2(taddr + c, taddr + c + 32, v[0], v[1]);
    }
    if (p.dw_tma) {
      if (lane == 0) bulk_wait_read<0>();  // the last store has read the tile
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 u;
        if (p.gf32) {
          u = make_uint4(__float_as_uint(v[0][4 * j]), __float_as_uint(v[0][4 * j + 1]), __float_as_uint(v[0][4 * j + 2]),
                         __float_as_uint(v[0][4 * j + 3]));
        } else {
          const float *s = &v[j >> 2][(j & 3) * 8];
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(s[2 * i], s[2 * i + 1]);
            w[i] = *(const uint32_t *)&b;
          }
          u = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *(uint4 *)(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = u;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (p.accumulate) tma_reduce_add_2d(&maps.dw, stg, col0 + c, row0);
        else tma_store_2d_hint(&maps.dw, stg, col0 + c, row0, out_policy);
        bulk_commit();
      }
    } else {
      by_rows(stg, v[0], lane, [&](int r, int cc, float4 x) {
        const int row = row0 + r, col = col0 + c + cc;
        if (row >= p.V) return;
        const float e[4] = {x.x, x.y, x.z, x.w};
        const int64_t at = (int64_t)row * p.D + col;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (col + j >= p.D) break;
          if (p.gf32) {
            float *o = (float *)p.dw + at + j;
            *o = p.accumulate ? *o + e[j] : e[j];
          } else {
            ((__nv_bfloat16 *)p.dw)[at + j] = __float2bfloat16_rn(e[j]);
          }
        }
      });
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(CtCfg<KIND>::THREADS, 1)
ce_pair_kernel(const __grid_constant__ CtMaps maps, const __grid_constant__ CtParams p) {
  constexpr int EPI_WARPS = CtCfg<KIND>::EPI_WARPS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *epi = base + CtCfg<KIND>::RING;
  uint64_t *bars = (uint64_t *)(epi + CtCfg<KIND>::STG_BYTES);
  uint64_t *full = bars, *empty = full + CT_MAX_STAGES;
  uint64_t *tfull = empty + CT_MAX_STAGES, *tempty = tfull + 2, *mma_done = tempty + 2;
  uint32_t *tmem_slot = (uint32_t *)(mma_done + 1);
  volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

  const int warp = __shfl_sync(FULL_MASK, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < CT_MAX_STAGES; ++s) {
      mbar_init(&full[s], 1);  // used in the even CTA
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (KIND == CE_GRADS) {
      prefetch_tmap(&maps.g);
      prefetch_tmap(p.w_blocks ? &maps.wt : &maps.wt1);
      prefetch_tmap(&maps.gt);
      prefetch_tmap(&maps.ht);
      if (p.dw_tma) prefetch_tmap(&maps.dw);
    } else {
      prefetch_tmap(&maps.h);
      prefetch_tmap(&maps.w);
      prefetch_tmap(&maps.h32);
      prefetch_tmap(&maps.w32);
      if (KIND == CE_LOGITS) prefetch_tmap(&maps.gout);
    }
  }
  cluster_sync();  // both CTAs' barriers exist before either touches the other's
  if (warp == 1) tmem_alloc_pair(tmem_slot, CT_TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, *tmem_slot, 0);
  griddep_launch();
  // With one row tile the weights are read once and nothing else counts: the
  // start of the pair's first tile is on its way into L2 (where later writes to it would
  // still be seen) while the kernels before this one finish.
  if (KIND == CE_STATS && p.tpad == CE_ROWS && warp == 2 && elect_one()) {
    const int units = (p.n + 63) / 64;
    const int u0 = (int)((int64_t)units * cid / ncl), u1 = (int)((int64_t)units * (cid + 1) / ncl);
    if (u1 - u0 >= 4)
      for (int k = 0; k < min(p.D, CT_PREFETCH * 64); k += 64) tma_prefetch_2d(&maps.w, k, p.v0 + u0 * 64 + (int)rank * 128);
  }
  griddep_wait();
  CtWork<KIND> work(p, cid, ncl);
  CtItem im;
  const int a_bytes = KIND != CE_GRADS && work.count <= 64 ? (work.count <= 32 ? 4096 : 8192) : CT_TILE;
  const int stages = min(CT_MAX_STAGES, CtCfg<KIND>::RING / (SUB * (a_bytes + CT_TILE)));
  auto sa = [&](int s, int j) { return base + (s * SUB + j) * (a_bytes + CT_TILE); };
  auto sb = [&](int s, int j) { return base + (s * SUB + j) * (a_bytes + CT_TILE) + a_bytes; };

  // The producers and the MMA issuer run their loops as whole warps, on values
  // that are the same in all lanes, and one elected lane issues: operands of
  // copies and MMAs then are in uniform registers from the start.  (Computed by a
  // single lane inside its branch, each copy took 410 cycles and each MMA 90.)
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers: A (warp 0), B (warp 2)
    const bool is_a = warp == 0, elected = elect_one();
    const uint64_t keep = policy_evict_last(), pass = policy_evict_first();
    // The weights' rows of a chunk are read by every row tile, those of one row tile once.
    const uint64_t wpol = work.mt > 1 ? keep : pass;
    const uint32_t full0 = mapa_shared(&full[0], 0);
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    bool ok = true;
    while (ok && work.next(p, im)) {
      const int mrow = im.m * 256 + (int)rank * 128;
      const int half = im.cols / 2, ncol = im.n0 + (int)rank * half;
      // Of the last rows only those that are there are read, 32 at a time: the
      // lines behind them reach nothing but accumulator rows that nobody reads.
      const int arows = KIND == CE_GRADS ? 128 : min(128, max(0, (work.count - mrow + 31) & ~31));
      const int arows2 = KIND == CE_GRADS ? 256 : min(256, max(0, (work.count - im.m * 256 + 31) & ~31));
      const uint32_t bytes = 128 * (arows2 + 2 * (uint32_t)half);
      for (int kb = 0; kb < im.nk; kb += SUB) {
        const int sub = min(SUB, im.nk - kb);
        if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) { ok = false; break; }
        const uint32_t bar = full0 + (uint32_t)(stage * sizeof(uint64_t));
        // Both CTAs' tiles complete on the even CTA's barrier.
        if (leader && is_a && elected) mbar_arrive_expect_tx(&full[stage], sub * bytes);
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          if (s >= sub) break;
          const int k = (kb + s) * 64;
          uint8_t *pa = sa(stage, s), *pb = sb(stage, s);
          if (!elected) continue;
          if (KIND != CE_GRADS) {
            if (is_a) {
              if (arows == 128) tma_load_2d_pair(pa, &maps.h, bar, k, mrow, keep);
              else
                for (int j = 0; j < arows; j += 32) tma_load_2d_pair(pa + j * 128, &maps.h32, bar, k, mrow + j, keep);
            } else {
              if (half == 128) tma_load_2d_pair(pb, &maps.w, bar, k, p.v0 + ncol, pass);
              else
                for (int j = 0; j < half; j += 32) tma_load_2d_pair(pb + j * 128, &maps.w32, bar, k, p.v0 + ncol + j, pass);
            }
          } else if (im.kind == 1) {
            const int v = im.chunk * p.chunk + k;
            if (is_a) tma_load_2d_pair(pa, &maps.g, bar, v, mrow, keep);
            else if (p.w_blocks && half == 128) tma_load_3d_pair(pb, &maps.wt, bar, 0, p.v0 + v, ncol / 64, wpol);
            else
              for (int j = 0; j < half; j += 64) tma_load_2d_pair(pb + j * 128, &maps.wt1, bar, ncol + j, p.v0 + v, wpol);
          } else {
            if (is_a) tma_load_3d_pair(pa, &maps.gt, bar, 0, k, mrow / 64, keep);
            else if (half == 128) tma_load_3d_pair(pb, &maps.ht, bar, 0, k, ncol / 64, keep);
            else tma_load_2d_pair(pb, &maps.ht1, bar, ncol, k, keep);
          }
        }
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) stage = 0, phase ^= 1;
      }
    }
    if (!ok) {
      // The copies in flight land before the pair exits: those that complete a
      // stage (both CTAs' do in the even CTA) are waited for, the others given the same time.
      volatile int never = 0;
      for (int s = 0; s < stages; ++s)
        if (issued & (1u << s)) mbar_wait(&full[s], (issued_phase >> s) & 1, &never, nullptr, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      // ---------------------------------------------------------- MMA issuer (both CTAs' tensor memory)
      const bool elected = elect_one();
      int stage = 0;
      uint32_t phase = 0, cnt = 0;
      bool ok = true;
      while (ok && work.next(p, im)) {
        if (im.nk == 0) continue;
        const bool a_mn = KIND == CE_GRADS && im.kind == 2, b_mn = KIND == CE_GRADS;
        const uint32_t idesc = idesc_bf16_f32(256, im.cols) | (a_mn ? IDESC_A_MN : 0) | (b_mn ? IDESC_B_MN : 0);
        const uint32_t astep = a_mn ? 128 : 2, bstep = b_mn ? 128 : 2;  // K = 16: 2048 or 32 bytes
        for (int kb = 0; kb < im.nk; kb += SUB) {
          const int kc = kb % CT_CHAIN<KIND>;  // in this accumulator
          const int sub = min(SUB, im.nk - kb);
          const int b = cnt & 1;
          if (kc == 0) {
            if (!warp_wait(&tempty[b], ((cnt >> 1) & 1) ^ 1, abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
          }
          if (!warp_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            if (s >= sub) break;
            const uint32_t a0 = smem_u32(sa(stage, s)), b0 = smem_u32(sb(stage, s));
            const uint64_t ad = a_mn ? smem_desc_mn_sw128(a0, 8192) : smem_desc_sw128(a0);
            const uint64_t bd = b_mn ? smem_desc_mn_sw128(b0, 8192) : smem_desc_sw128(b0);
            if (elected) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_pair(tmem + b * 256, ad + astep * kk, bd + bstep * kk, idesc, (kc | s | kk) != 0);
            }
          }
          const bool last = kb + sub == im.nk || kc + sub == CT_CHAIN<KIND>;
          if (elected) {
            mma_commit_pair(&empty[stage]);
            if (last) mma_commit_pair(&tfull[b]);
          }
          __syncwarp();
          if (last) ++cnt;
          if (++stage == stages) stage = 0, phase ^= 1;
        }
      }
      if (elected) mma_commit_pair(mma_done);
      __syncwarp();
    }
    // Every pair MMA has finished (it wrote both CTAs' tensor memory) before TMEM is released.
    volatile int never = 0;
    if (lane == 0) ct_wait(mma_done, 0, &never, p.status);
    __syncwarp();
  } else if (warp >= CT_EPI_FIRST) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - CT_EPI_FIRST) >> 2;  // TMEM lane quarter; which of the columns
    uint8_t *stg = epi + (warp - CT_EPI_FIRST) * CtCfg<KIND>::STG_WARP;
    const uint32_t tempty_leader0 = mapa_shared(&tempty[0], 0);
    const uint64_t out_policy = policy_evict_first();  // dweight is written once and not read again
    uint32_t cnt = 0;
    auto wait = [&] {
      if (!warp_wait(&tfull[cnt & 1], (cnt >> 1) & 1, abort_flag, p.status)) return false;
      tc_fence_after();
      return true;
    };
    auto release = [&](uint32_t b) {  // an accumulator, to the MMA thread
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(&tempty[b]);
        else mbar_arrive_remote(tempty_leader0 + (uint32_t)(b * sizeof(uint64_t)));
      }
    };
    // A sum that goes on: what it has come to, onto its next part (this warp's columns).
    auto carry = [&](uint32_t from, uint32_t to) {
#pragma unroll 1
      for (int c = half * (im.cols / 2); c < (half + 1) * (im.cols / 2); c += 32) {
        float a[32], b[32];
        tmem_ld32x2(from + c, to + c, a, b);
#pragma unroll
        for (int j = 0; j < 32; ++j) b[j] += a[j];
        tmem_st32(to + c, b);
      }
    };
    while (work.next(p, im)) {
      const int row0 = im.m * 256 + (int)rank * 128 + q * 32;
      const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
      if (KIND != CE_GRADS) {
        float v[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = 0.f;
        bool ok = true;
        for (int kb = 0; kb < im.nk; kb += CT_KCHUNK) {
          if (!(ok = wait())) break;
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            if (half * 64 >= im.cols) break;
            float x[16];
            tmem_ld16(tq + (cnt & 1) * 256 + half * 64 + c, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[c + j] += x[j];
          }
          release(cnt & 1);
          ++cnt;
        }
        if (!ok) break;
        if (KIND == CE_STATS) stats_epilogue(p, im, v, row0 + lane, half);
        else logits_epilogue(maps, p, im, v, row0 + lane, half, stg, lane);
        continue;
      }
      bool ok = true;
      for (int kb = 0; kb < im.nk; kb += CT_CHAIN<KIND>) {
        if (!(ok = wait())) break;
        if (kb != 0) {
          carry(tq + (~cnt & 1) * 256, tq + (cnt & 1) * 256);
          release(~cnt & 1);
        }
        if (kb + CT_CHAIN<KIND> < im.nk) ++cnt;
      }
      if (!ok) break;
      const uint32_t taddr = tq + (cnt & 1) * 256 + half * (im.cols / 2);
      if (im.kind == 1) dhidden_epilogue(p, im, taddr, row0, work.count, half, stg, lane);
      else dweight_epilogue(maps, p, im, taddr, p.v0 + row0, half, stg, lane, out_policy);
      if (im.nk != 0) {
        release(cnt & 1);
        ++cnt;
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no remote arrival, copy or commit targets this CTA any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, CT_TMEM_COLS);
}

// ------------------------------------------------------------------ host side
// Row-major [rows, cols] of bf16 (or float) with a row stride of ld elements.
static bool map_ld(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows,
                   bool f32 = false) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)ld * (f32 ? 4 : 2)};
  const uint32_t box[2] = {f32 ? 32u : 64u, box_rows};
  return encode_map(m, ptr, 2, dims, strides, box, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

// The same (cols % 64 == 0) in blocks of 64 columns: boxes of 64 rows x 64 x 2.
static bool map_blocks(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t ld) {
  const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64};
  const uint64_t strides[2] = {(uint64_t)ld * 2, 128};
  const uint32_t box[3] = {64, 64, 2};
  return encode_map(m, ptr, 3, dims, strides, box);
}

template <int KIND>
static cudaError_t launch(const CtMaps &maps, const CtParams &p, int64_t items, cudaStream_t stream) {
  cudaError_t e = ensure_smem((const void *)ce_pair_kernel<KIND>, CtCfg<KIND>::SMEM);
  if (e != cudaSuccess) return e;
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(items, device_sms() / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(CtCfg<KIND>::THREADS);
  cfg.dynamicSmemBytes = CtCfg<KIND>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ce_pair_kernel<KIND>, maps, p);
}

static CtParams params(const CeMats &m) {
  CtParams p = {};
  p.V = m.V;
  p.D = m.D;
  p.tpad = m.tpad;
  p.count = m.count;
  p.row_of = m.row_of;
  p.rows = m.rows;
  p.inv = m.inv;
  p.s2 = m.scale * CE_LOG2E;
  p.part = m.part;
  p.xt = m.xt;
  p.n = m.V;
  p.ldh = m.ldh;
  p.status = m.status;
  return p;
}

static void piece(CtParams &p, const CePiece &c) {
  p.v0 = c.v0;
  p.n = c.n;
  p.chunk = c.chunk;
  p.nchunks = c.nchunks;
  p.first = c.first;
  p.last = c.last;
}

cudaError_t ce_tc_stats(const CeMats &m, cudaStream_t stream) {
  CtMaps maps = {};
  if (!map_ld(&maps.h, m.h, m.tpad, m.ldh, m.ldh, 128) || !map_ld(&maps.h32, m.h, m.tpad, m.ldh, m.ldh, 32) ||
      !map_ld(&maps.w, m.w, m.V, m.D, m.ldw, 128) ||
      !map_ld(&maps.w32, m.w, m.V, m.D, m.ldw, 32))
    return cudaErrorInvalidValue;
  return launch<CE_STATS>(maps, params(m), (int64_t)(m.tpad / 256) * ceil_div(m.V, 64), stream);
}

cudaError_t ce_tc_logits_grad(const CeMats &m, const CePiece &c, cudaStream_t stream) {
  CtMaps maps = {};
  CtParams p = params(m);
  piece(p, c);
  const uint64_t gdims[2] = {(uint64_t)m.ldg, (uint64_t)m.tpad}, gstride[1] = {(uint64_t)m.ldg * 2};
  const uint32_t gbox[2] = {32, 32};
  if (!map_ld(&maps.h, m.h, m.tpad, m.ldh, m.ldh, 128) || !map_ld(&maps.h32, m.h, m.tpad, m.ldh, m.ldh, 32) ||
      !map_ld(&maps.w, m.w, m.V, m.D, m.ldw, 128) ||
      !map_ld(&maps.w32, m.w, m.V, m.D, m.ldw, 32) ||
      !encode_map(&maps.gout, m.g, 2, gdims, gstride, gbox, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  return launch<CE_LOGITS>(maps, p, (int64_t)(m.tpad / 256) * ceil_div(c.n, 64), stream);
}

cudaError_t ce_tc_grads(const CeMats &m, const CePiece &c, cudaStream_t stream) {
  CtMaps maps = {};
  CtParams p = params(m);
  piece(p, c);
  p.accumulate = m.accumulate;
  p.gf32 = m.gf32;
  p.dw = m.dw;
  p.dh = (__nv_bfloat16 *)m.dh;
  p.ld_dh = m.ld_dh;
  p.dh_wide = m.D % 4 == 0 && m.ld_dh % 4 == 0 && ((uintptr_t)m.dh & 7) == 0;
  p.acc = m.acc;
  p.planes = m.planes;
  p.w_blocks = m.D % 64 == 0;
  // Tensor maps of dweight want its dense rows on 16-byte boundaries.
  p.dw_tma = ((uintptr_t)m.dw & 15) == 0 && m.D % (m.gf32 ? 4 : 8) == 0;
  if (!map_ld(&maps.g, m.g, m.tpad, m.ldg, m.ldg, 128) || !map_blocks(&maps.gt, m.g, m.tpad, m.ldg, m.ldg) ||
      (p.w_blocks && !map_blocks(&maps.wt, m.w, m.V, m.D, m.ldw)) || !map_ld(&maps.wt1, m.w, m.V, m.D, m.ldw, 64) ||
      !map_blocks(&maps.ht, m.h2, m.tpad, m.ldh, m.ldh) || !map_ld(&maps.ht1, m.h2, m.tpad, m.ldh, m.ldh, 64) ||
      (p.dw_tma && !map_ld(&maps.dw, m.dw, m.V, m.D, m.D, 32, m.gf32)))
    return cudaErrorInvalidValue;
  const int64_t nt = ceil_div(m.D, 256);
  return launch<CE_GRADS>(maps, p, nt * ((int64_t)c.nchunks * (m.tpad / 256) + ceil_div(c.n, 256)), stream);
}

}  // namespace moe

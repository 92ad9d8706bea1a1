// Token embedding with a scale, and its gradient by sorted tokens (contracts
// with moe_embed in moe.h).
//
// Lookup: groups of threads take four rows each and have all four on their
// way before the first is written; it moves the rows read and written once.
//
// Gradient:
//   1. the tokens are sorted, stable, by two counting passes over half of a
//      token's bits each: one launch on a cluster of sixteen CTAs, whose
//      counts meet in distributed shared memory (for more tokens than that is
//      good for, the kernels of the route permutation, twice);
//   2. meanwhile, on the other SMs, the rows of the table that no token hits
//      are zeroed;
//   3. tiles of consecutive sorted positions sum their rows, token by token.
//      A token that lies in one tile is written at once, one that spans tiles
//      leaves a partial row in each;
//   4. the partial rows of such a token are added in order.
// Tokens left out (outside the table, or the padding token) sort behind the
// table as token V.  A tile's bounds depend on the number of tokens alone.
//
// The gradient's floor is its rows read once and the table written once: 198 us
// for 65536 tokens into 131072 x 2048, 43.5 us for 4096 float rows into
// 32000 x 2048.  Measured: 271 us (73 %) and 59 us (73 %), of which the zeroing,
// at the rate of memory, takes 144 and 40, the sums 80 and 13, the joins 28 and
// 9; the sort (27 and 13) hides behind the zeroing.  Reached from 5445 us (the
// permutation's sort twice, a CTA a row of the table): tiles and joins 339,
// only rows without a token zeroed and longer loads in the sums 314, spans
// listed and joined by warps 273.  The lookup of 16384 rows of 2048 takes
// 19 us of which 14 are its floor.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int EM_THREADS = 256, EM_ROWS = 4;
constexpr int ES_CTAS = 16, ES_THREADS = 1024, ES_WARPS = 32;
constexpr int EM_DIGIT = 1024;                   // of the permutation's kernels
constexpr int ES_STEPS = 8;                      // of 32 positions a warp
constexpr int64_t ES_MAX_T = ES_CTAS * ES_WARPS * 32 * ES_STEPS;  // tokens of the one-launch sort

__device__ inline int64_t em_id(const EmbedArgs &a, int64_t t) {
  return a.ids64 ? ((const int64_t *)a.ids)[t] : (int64_t)((const int32_t *)a.ids)[t];
}
// The sort key of token t: its row of the table, V where it is left out.
__device__ inline int32_t em_key(const EmbedArgs &a, int64_t t, int *status) {
  const int64_t id = em_id(a, t);
  const bool ok = id >= 0 && id < a.V;
  if (!ok) record_status(status, STATUS_BAD_TOKEN_ID);
  return ok && id != a.padding_id ? (int32_t)id : a.V;
}

// What a thread holds of a row: VEC neighbouring elements, or, where rows do
// not all start on 16-byte boundaries (VEC = 0), four elements `stride` apart.
template <int VEC>
constexpr int em_n() {
  return VEC ? VEC : 4;
}
template <typename T, int VEC>
__device__ inline void em_load(const T *row, int i, int stride, int H, float (&o)[em_n<VEC>()]) {
  if constexpr (VEC == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = i + k * stride < H ? Elem<T>::load(row + i + k * stride) : 0.f;
  } else {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int b = 0; b < VEC / N; ++b) {
      float v[N];
      Vec16<T>::load(row + i + b * N, v);
#pragma unroll
      for (int k = 0; k < N; ++k) o[b * N + k] = v[k];
    }
  }
}
template <typename T, int VEC>
__device__ inline void em_store(T *row, int i, int stride, int H, const float (&v)[em_n<VEC>()]) {
  if constexpr (VEC == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * stride < H) row[i + k * stride] = Elem<T>::from_f32(v[k]);
  } else {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int b = 0; b < VEC / N; ++b) {
      float o[N];
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = v[b * N + k];
      Vec16<T>::store(row + i + b * N, o);
    }
  }
}

// ---------------------------------------------------------------- lookup
template <typename TE, typename TO, int VEC>
__global__ void __launch_bounds__(EM_THREADS, 4) embed_kernel(const EmbedArgs a, int group, int rows, int *status) {
  constexpr int N = em_n<VEC>();
  griddep_launch();
  griddep_wait();
  const int per_cta = EM_THREADS / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const int64_t step = (int64_t)gridDim.x * per_cta * rows;
  int64_t t0 = ((int64_t)blockIdx.x * per_cta + sub) * rows;
  int64_t next[EM_ROWS];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int r = 0; r < EM_ROWS; ++r) next[r] = r < rows && t + r < a.T ? em_id(a, t + r) : 0;
  };
  fetch(t0);
  for (; t0 < a.T; t0 += step) {
    const TE *src[EM_ROWS];
#pragma unroll
    for (int r = 0; r < EM_ROWS; ++r) {
      src[r] = nullptr;
      if (r < rows && t0 + r < a.T) {
        if (next[r] >= 0 && next[r] < a.V) src[r] = (const TE *)a.table + next[r] * a.ld_table;
        else if (lane == 0) record_status(status, STATUS_BAD_TOKEN_ID);
      }
    }
    fetch(t0 + step);
    for (int i = VEC ? lane * VEC : lane; i < a.H; i += group * N) {
      float v[EM_ROWS][N];
#pragma unroll
      for (int r = 0; r < EM_ROWS; ++r) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[r][k] = 0.f;
        if (src[r]) em_load<TE, VEC>(src[r], i, group, a.H, v[r]);
      }
#pragma unroll
      for (int r = 0; r < EM_ROWS; ++r)
        if (r < rows && t0 + r < a.T) {
#pragma unroll
          for (int k = 0; k < N; ++k) v[r][k] *= a.scale;
          em_store<TO, VEC>((TO *)a.out + (t0 + r) * a.ld_out, i, group, a.H, v[r]);
        }
    }
  }
}

// ---------------------------------------------------------------- sort
__device__ inline int32_t es_ld_cluster(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Two stable counting passes over `bits` bits each.  CTA c takes the c-th
// sixteenth of the positions, warp w a contiguous part of it; a warp's counts
// are prefixed over warps, CTAs and digits, then its positions are handed out
// in order, 32 at a time.  Buffers hold T entries.
__global__ void __launch_bounds__(ES_THREADS)
embed_sort_kernel(const EmbedArgs a, int bits, int32_t *mark, int32_t *key1, int32_t *pos1, int32_t *key2, int32_t *pos2,
                  int32_t *spans, int *status) {
  using namespace umma;
  extern __shared__ int32_t es_smem[];
  const int D = 1 << bits;
  int32_t *hist = es_smem, *total = hist + ES_WARPS * D, *wsum = total + D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  griddep_wait();
  const int T = a.T;
  const int per_warp = (int)round_up(ceil_div(T, ES_CTAS * ES_WARPS), 32);
  const int begin = (rank * ES_WARPS + warp) * per_warp, end = min(begin + per_warp, T);
  int32_t *mine = hist + warp * D;
  for (int pass = 0; pass < 2; ++pass) {
    // The warp's positions, 32 at a time.
    int32_t keys[ES_STEPS], tokens[ES_STEPS];
#pragma unroll
    for (int q = 0; q < ES_STEPS; ++q) {
      const int j = begin + 32 * q + lane;
      keys[q] = tokens[q] = -1;
      if (j < end) {
        keys[q] = pass ? ld_l2(key1 + j) : em_key(a, j, status);
        tokens[q] = pass ? ld_l2(pos1 + j) : j;
      }
    }
    for (int d = threadIdx.x; d < ES_WARPS * D; d += ES_THREADS) hist[d] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < ES_STEPS; ++q)
      if (keys[q] >= 0) {
        atomicAdd(mine + ((keys[q] >> (pass * bits)) & (D - 1)), 1);
        if (pass == 0 && keys[q] < a.V) mark[keys[q]] = tokens[q];
      }
    if (pass == 0 && rank == 0 && threadIdx.x == 0) *spans = 0;
    if (pass == 0) griddep_launch();  // the zeroing may start: what came before this kernel has finished
    __syncthreads();
    // Before this warp in the CTA.
    const int d = threadIdx.x;
    int32_t sum = 0;
    if (d < D) {
      for (int w = 0; w < ES_WARPS; ++w) {
        const int32_t n = hist[w * D + d];
        hist[w * D + d] = sum;
        sum += n;
      }
      total[d] = sum;
    }
    cluster_sync();
    // Of this digit in all CTAs, and in those before this one.
    int32_t all = 0, before = 0;
    if (d < D) {
      int32_t n[ES_CTAS];
#pragma unroll
      for (int c = 0; c < ES_CTAS; ++c) n[c] = es_ld_cluster(mapa_shared(total + d, c));
#pragma unroll
      for (int c = 0; c < ES_CTAS; ++c) {
        all += n[c];
        if (c < rank) before += n[c];
      }
    }
    // Of the digits before it (exclusive scan over the block).
    int32_t inc = all;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int32_t u = __shfl_up_sync(FULL_MASK, inc, s);
      if (lane >= s) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    cluster_sync();  // (the others have read this CTA's totals)
    if (warp == 0) {
      int32_t v = wsum[lane], x = v;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int32_t u = __shfl_up_sync(FULL_MASK, x, s);
        if (lane >= s) x += u;
      }
      wsum[lane] = x - v;
    }
    __syncthreads();
    if (d < D) total[d] = wsum[warp] + inc - all + before;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < ES_STEPS; ++q) {
      if (begin + 32 * q >= end) break;
      const bool in = keys[q] >= 0;
      const int digit = in ? (keys[q] >> (pass * bits)) & (D - 1) : -1 - lane;
      const unsigned same = __match_any_sync(FULL_MASK, digit);
      const int ahead = __popc(same & lanemask_lt());
      int32_t base = 0;
      if (in) base = total[digit] + mine[digit];
      __syncwarp();
      if (in && ahead == 0) mine[digit] += __popc(same);
      __syncwarp();
      if (in) {
        (pass ? key2 : key1)[base + ahead] = keys[q];
        (pass ? pos2 : pos1)[base + ahead] = tokens[q];
      }
    }
    if (pass == 0) {
      __threadfence();
      cluster_sync();
    }
  }
}

// The same by the permutation's kernels: low digits, then high digits.
__global__ void __launch_bounds__(256) embed_key_kernel(const EmbedArgs a, int32_t *key, int32_t *lo, int32_t *spans, int *status) {
  griddep_launch();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *spans = 0;
  for (int64_t t = blockIdx.x * 256ll + threadIdx.x; t < a.T; t += gridDim.x * 256ll) {
    const int32_t k = em_key(a, t, status);
    key[t] = k;
    lo[t] = k & (EM_DIGIT - 1);
  }
}
__global__ void __launch_bounds__(256) embed_high_kernel(int64_t T, const int32_t *key, const int32_t *first,
                                                         int32_t *hi) {
  griddep_launch();
  griddep_wait();
  for (int64_t j = blockIdx.x * 256ll + threadIdx.x; j < T; j += gridDim.x * 256ll) hi[j] = key[first[j]] / EM_DIGIT;
}
__global__ void __launch_bounds__(256) embed_order_kernel(int64_t T, const int32_t *key, const int32_t *first,
                                                          const int32_t *second, int32_t *skey, int32_t *order) {
  griddep_launch();
  griddep_wait();
  for (int64_t j = blockIdx.x * 256ll + threadIdx.x; j < T; j += gridDim.x * 256ll) {
    const int t = first[second[j]];
    order[j] = t;
    skey[j] = key[t];
  }
}

// ---------------------------------------------------------------- zeroing
// Zeroes dtable.  With `mark` it runs beside the one-launch sort, which lets it
// start once what came before has finished; it waits for the sort at its end
// only, so that what follows waits for both.  mark[v] is a token of row v or
// not written: a row whose mark is such a token is written by the sums and
// left alone here (one that were zeroed all the same would only be written
// twice).  A warp takes `rows` rows at a time, at most 32.
__global__ void __launch_bounds__(512) embed_zero_kernel(const EmbedArgs a, const int32_t *mark, int rows) {
  if (!mark) griddep_wait();
  const int lane = threadIdx.x & 31;
  const bool wide = a.H % 4 == 0 && ((uintptr_t)a.dtable & 15) == 0;
  const int64_t step = (int64_t)gridDim.x * 16 * rows;
  for (int64_t v0 = ((int64_t)blockIdx.x * 16 + (threadIdx.x >> 5)) * rows; v0 < a.V; v0 += step) {
    bool hit = lane >= rows || v0 + lane >= a.V;
    if (mark && !hit) {
      const int32_t t = ld_l2(mark + v0 + lane);
      if (t >= 0 && t < a.T) {
        const int64_t id = em_id(a, t);
        hit = id == v0 + lane && id != a.padding_id;
      }
    }
    for (unsigned left = ~__ballot_sync(FULL_MASK, hit); left; left &= left - 1) {
      float *row = a.dtable + (v0 + __ffs(left) - 1) * a.H;
      if (wide) {
        for (int i = lane; i < a.H / 4; i += 32) __stcs((float4 *)row + i, make_float4(0.f, 0.f, 0.f, 0.f));
      } else {
        for (int i = lane; i < a.H; i += 32) __stcs(row + i, 0.f);
      }
    }
  }
  if (mark) griddep_wait();
}

// ---------------------------------------------------------------- sums
// Tiles of `tile` sorted positions; part: [tiles][2][H], a tile's sums of the
// token that was there before it (0) and of the one that goes on behind it (1).
template <typename TO, int VEC>
__global__ void __launch_bounds__(EM_THREADS)
embed_sum_kernel(const EmbedArgs a, int tile, int group, const int32_t *key, const int32_t *order, float *part,
                 int32_t *spans, int32_t *span_tiles) {
  constexpr int AHEAD = 8, N = em_n<VEC>();
  // Keys and tokens of the CTA's tiles.
  __shared__ int32_t skey[EM_THREADS], sorder[EM_THREADS];
  griddep_launch();
  griddep_wait();
  const int per_cta = EM_THREADS / group, sub = threadIdx.x / group, lane = threadIdx.x % group;
  const int64_t b = (int64_t)blockIdx.x * per_cta + sub;
  const int64_t start = (int64_t)blockIdx.x * per_cta * tile;
  const int p0 = (int)min(b * tile, (int64_t)a.T), p1 = min(p0 + tile, a.T);
  const int i = blockIdx.y * group * N + (VEC ? lane * VEC : lane);
  const bool live = p0 < p1 && i < a.H;
  const int first = live ? key[p0] : a.V;
  const int after = live && p1 < a.T ? key[p1] : a.V;
  bool before = live && p0 > 0 && key[p0 - 1] == first;  // whether the token was there before this tile
  float s[N];
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = 0.f;
  int now = first;
  auto flush = [&](bool goes_on) {
    if (before || goes_on) {
      em_store<float, VEC>(part + (b * 2 + (before ? 0 : 1)) * a.H, i, group, a.H, s);
      if (!before && lane == 0 && blockIdx.y == 0) span_tiles[atomicAdd(spans, 1)] = (int32_t)b;
    } else {
      float *o = a.dtable + (int64_t)now * a.H;
      float v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = 0.f;
      if (a.accumulate) em_load<float, VEC>(o, i, group, a.H, v);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = a.accumulate ? fmaf(a.scale, s[k], v[k]) : a.scale * s[k];
      em_store<float, VEC>(o, i, group, a.H, v);
    }
  };
  // Rounds of n positions of each tile, so many that all tiles' fit.
  const int n = min(tile, EM_THREADS / per_cta);
  for (int q = 0; q < tile; q += n) {
    __syncthreads();
    {
      const int64_t at = start + (int64_t)(threadIdx.x / n) * tile + q + threadIdx.x % n;
      if ((int)threadIdx.x < n * per_cta && at < a.T) {
        skey[threadIdx.x] = key[at];
        sorder[threadIdx.x] = order[at];
      }
    }
    __syncthreads();
    const int m = min(n, p1 - p0 - q), at = sub * n;
    for (int p = 0; p < m && now < a.V; p += AHEAD) {
      uint4 raw[VEC ? AHEAD : 1];
      TO loose[VEC ? 1 : AHEAD][4];
#pragma unroll
      for (int r = 0; r < AHEAD; ++r)
        if (p + r < m && skey[at + p + r] < a.V) {
          const TO *row = (const TO *)a.dout + (int64_t)sorder[at + p + r] * a.ld_out;
          if constexpr (VEC != 0) {
            static_assert(VEC == Vec16<TO>::N, "one 16-byte load");
            raw[r] = ld_once((const uint4 *)(row + i));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (i + k * group < a.H) loose[r][k] = row[i + k * group];
          }
        }
#pragma unroll
      for (int r = 0; r < AHEAD; ++r) {
        if (p + r >= m || now >= a.V) break;
        const int k_at = skey[at + p + r];
        if (k_at != now) {
          flush(false);
          before = false;
          now = k_at;
#pragma unroll
          for (int k = 0; k < N; ++k) s[k] = 0.f;
          if (now >= a.V) break;
        }
        float v[N];
        if constexpr (VEC != 0) {
          Vec16<TO>::unpack(raw[r], v);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = i + k * group < a.H ? Elem<TO>::to_f32(loose[r][k]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += v[k];
      }
    }
  }
  if (now < a.V) flush(after == now);
}

// Tokens that span tiles, listed by the tile that each starts in: a warp adds
// the partial rows of one up, in order, 32 channels at a time.
__global__ void __launch_bounds__(EM_THREADS, 4) embed_join_kernel(const EmbedArgs a, int tile, const int32_t *key,
                                                                   const float *part, const int32_t *spans,
                                                                   const int32_t *span_tiles) {
  constexpr int AHEAD = 16;  // a join is a chain of loads: many at a time
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, slices = (a.H + 31) / 32;
  const int64_t tiles = ceil_div(a.T, tile), items = (int64_t)*spans * slices, warps = (int64_t)gridDim.x * (EM_THREADS / 32);
  for (int64_t w = (int64_t)blockIdx.x * (EM_THREADS / 32) + (threadIdx.x >> 5); w < items; w += warps) {
    const int64_t b = span_tiles[w / slices];
    const int i = (int)(w % slices) * 32 + lane;
    const int32_t now = key[(b + 1) * tile];
    int64_t n = 1;  // tiles behind that one which it reaches
    for (;;) {
      const int64_t c = b + 1 + n + lane;
      const int got = __popc(__ballot_sync(FULL_MASK, c < tiles && key[c * tile] == now));
      n += got;
      if (got < 32) break;
    }
    if (i >= a.H) continue;
    float s = part[(b * 2 + 1) * a.H + i];
    const float *q = part + (b + 1) * 2 * (int64_t)a.H + i;
    for (int64_t c = 0; c < n; c += AHEAD) {
      float v[AHEAD];
#pragma unroll
      for (int r = 0; r < AHEAD; ++r) v[r] = c + r < n ? q[(c + r) * 2 * a.H] : 0.f;
#pragma unroll
      for (int r = 0; r < AHEAD; ++r) s += v[r];
    }
    float *o = a.dtable + (int64_t)now * a.H + i;
    *o = a.accumulate ? fmaf(a.scale, s, *o) : a.scale * s;
  }
}

// ---------------------------------------------------------------- host
static bool em_wide(const void *p, int64_t ld, int es, int H, int vec) {
  return H % vec == 0 && ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0;
}
// Threads that share a row of H elements: a power of two.
static int em_group(int H, int vec) {
  int g = 1;
  while (g < EM_THREADS && g * vec < H) g *= 2;
  return g;
}

template <typename TE, typename TO>
static cudaError_t embed_types(const EmbedArgs &a, int *status, cudaStream_t stream) {
  constexpr int VEC = Vec16<TE>::N;
  const bool wide = em_wide(a.table, a.ld_table, sizeof(TE), a.H, VEC) && em_wide(a.out, a.ld_out, sizeof(TO), a.H, VEC);
  const int group = em_group(a.H, wide ? VEC : 4);
  // Four rows a group where there are enough of them to fill the SMs.
  const int rows = ceil_div(a.T, EM_THREADS / group) >= (int64_t)device_sms() * 2 * EM_ROWS ? EM_ROWS : 1;
  const int64_t ctas = ceil_div(a.T, (int64_t)(EM_THREADS / group) * rows);
  const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)device_sms() * 4)), block(EM_THREADS);
  if (wide) return launch_pdl(embed_kernel<TE, TO, VEC>, grid, block, 0, stream, a, group, rows, status);
  return launch_pdl(embed_kernel<TE, TO, 0>, grid, block, 0, stream, a, group, rows, status);
}

cudaError_t launch_embed(const EmbedArgs &a, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  if (a.f32) return embed_types<float, float>(a, status, stream);
  if (a.of32) return embed_types<__nv_bfloat16, float>(a, status, stream);
  return embed_types<__nv_bfloat16, __nv_bfloat16>(a, status, stream);
}

// Sorted positions of a tile: enough tiles to fill the SMs, few enough partial rows.
static int em_tile(int T) { return T < 16384 ? 8 : T < 65536 ? 16 : T < (1 << 18) ? 32 : T < (1 << 20) ? 64 : 256; }

// Whether the cluster of the one-launch sort fits the current device.
static bool es_fits() {
  static std::mutex mu;
  static int known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  int &k = known[dev & 63];
  if (!k) {
    const int smem = ((ES_WARPS + 1) * EM_DIGIT + 64) * 4;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ES_CTAS);
    cfg.blockDim = dim3(ES_THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ES_CTAS;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const bool ok = ensure_smem((const void *)embed_sort_kernel, smem) == cudaSuccess &&
                    cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, embed_sort_kernel, &cfg) == cudaSuccess && n >= 1;
    if (!ok) cudaGetLastError();  // not an error of the caller's
    k = ok ? 1 : 2;
  }
  return k == 1;
}

static bool es_used(const EmbedArgs &a) { return a.T <= ES_MAX_T && es_fits(); }

struct EmbedScratch {
  int32_t *key, *order, *key1, *pos1, *mark, *spans, *span_tiles, *lo, *second, *digits;
  float *part;
  void *sort;
};
static EmbedScratch embed_carve(const EmbedArgs &a, char *base, size_t *bytes) {
  size_t off = 0;
  auto take = [&](size_t n) {
    char *p = base + off;
    off += (n + 255) / 256 * 256;
    return p;
  };
  EmbedScratch s = {};
  const size_t t = (size_t)a.T * 4;
  s.key = (int32_t *)take(t);
  s.order = (int32_t *)take(t);
  s.key1 = (int32_t *)take(t);
  s.pos1 = (int32_t *)take(t);
  s.part = (float *)take((size_t)ceil_div(a.T, em_tile(a.T)) * 2 * a.H * 4);
  s.mark = (int32_t *)take((size_t)a.V * 4);
  s.spans = (int32_t *)take(4);
  s.span_tiles = (int32_t *)take((size_t)ceil_div(a.T, em_tile(a.T)) * 4);
  s.lo = (int32_t *)take(t);
  s.second = (int32_t *)take(t);
  s.digits = (int32_t *)take((EM_DIGIT + 1) * 4);
  s.sort = take(permute_scratch_bytes(a.T, EM_DIGIT));
  *bytes = off;
  return s;
}

size_t embed_scratch_bytes(const EmbedArgs &a) {
  size_t n;
  embed_carve(a, nullptr, &n);
  return n;
}

static cudaError_t embed_sort(const EmbedArgs &a, const EmbedScratch &s, int *status, cudaStream_t stream) {
  if (es_used(a)) {
    int bits = 1;  // half of the bits of a key (V among them)
    while ((int64_t)a.V >> (2 * bits)) ++bits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ES_CTAS);
    cfg.blockDim = dim3(ES_THREADS);
    cfg.dynamicSmemBytes = ((ES_WARPS + 1) * (1 << bits) + 64) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ES_CTAS;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a, bits, s.mark, s.key1, s.pos1, s.key, s.order, s.spans, status);
  }
  const int64_t T = a.T;
  const dim3 grid((unsigned)ceil_div(T, 256)), block(256);
  cudaError_t e = launch_pdl(embed_key_kernel, grid, block, 0, stream, a, s.key1, s.lo, s.spans, status);
  if (e == cudaSuccess) e = launch_permute(T, EM_DIGIT, s.lo, s.digits, s.pos1, s.key, s.sort, status, stream);
  if (e == cudaSuccess)
    e = launch_pdl(embed_high_kernel, grid, block, 0, stream, T, (const int32_t *)s.key1, (const int32_t *)s.pos1, s.lo);
  if (e == cudaSuccess) e = launch_permute(T, EM_DIGIT, s.lo, s.digits, s.second, s.key, s.sort, status, stream);
  if (e == cudaSuccess)
    e = launch_pdl(embed_order_kernel, grid, block, 0, stream, T, (const int32_t *)s.key1, (const int32_t *)s.pos1,
                   (const int32_t *)s.second, s.key, s.order);
  return e;
}

template <typename TO>
static cudaError_t embed_sum(const EmbedArgs &a, const EmbedScratch &s, cudaStream_t stream) {
  constexpr int VEC = Vec16<TO>::N;
  const bool wide = em_wide(a.dout, a.ld_out, sizeof(TO), a.H, VEC) && em_wide(a.dtable, a.H, 4, a.H, VEC);
  const int vec = wide ? VEC : 4, group = em_group(a.H, vec), tile = em_tile(a.T);
  const int64_t tiles = ceil_div(a.T, tile);
  const dim3 grid((unsigned)ceil_div(tiles, EM_THREADS / group), (unsigned)ceil_div(a.H, group * vec));
  const int32_t *key = s.key, *order = s.order;
  cudaError_t e = wide ? launch_pdl(embed_sum_kernel<TO, VEC>, grid, dim3(EM_THREADS), 0, stream, a, tile, group, key, order, s.part, s.spans, s.span_tiles)
                       : launch_pdl(embed_sum_kernel<TO, 0>, grid, dim3(EM_THREADS), 0, stream, a, tile, group, key, order, s.part, s.spans, s.span_tiles);
  if (e != cudaSuccess || tiles < 2) return e;
  const int64_t warps = tiles * ceil_div(a.H, 32);  // at most
  return launch_pdl(embed_join_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(warps, EM_THREADS / 32), (int64_t)device_sms() * 4)),
                    dim3(EM_THREADS), 0, stream, a, tile, key, (const float *)s.part, (const int32_t *)s.spans,
                    (const int32_t *)s.span_tiles);
}

cudaError_t launch_embed_bwd(const EmbedArgs &a, void *scratch, int *status, cudaStream_t stream) {
  const int64_t n = (int64_t)a.V * a.H;
  if (a.T == 0) return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.dtable, 0, (size_t)n * sizeof(float), stream);
  size_t bytes;
  const EmbedScratch s = embed_carve(a, (char *)scratch, &bytes);
  cudaError_t e = embed_sort(a, s, status, stream);
  if (e == cudaSuccess && !a.accumulate) {
    const int rows = std::max(1, std::min(32, 4096 / a.H));
    const int64_t ctas = std::min<int64_t>(ceil_div(a.V, 16 * rows), (int64_t)device_sms() * 4);
    e = launch_pdl(embed_zero_kernel, dim3((unsigned)ctas), dim3(512), 0, stream, a, (const int32_t *)(es_used(a) ? s.mark : nullptr), rows);
  }
  if (e != cudaSuccess) return e;
  return a.of32 ? embed_sum<float>(a, s, stream) : embed_sum<__nv_bfloat16>(a, s, stream);
}

}  // namespace moe

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
//   2. meanwhile, on the other SMs, the table is zeroed;
//   3. tiles of consecutive sorted positions sum their rows, token by token.
//      A token that lies in one tile is written at once, one that spans tiles
//      leaves a partial row in each;
//   4. the partial rows of such a token are added in order.
// Tokens left out (outside the table, or the padding token) sort behind the
// table as token V.  A tile's bounds depend on the number of tokens alone.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int EM_THREADS = 256, EM_ROWS = 4;
constexpr int ES_CTAS = 16, ES_THREADS = 1024, ES_WARPS = 32;
constexpr int EM_DIGIT = 1024;                   // of the permutation's kernels
constexpr int64_t ES_MAX_T = int64_t(1) << 17;   // tokens of the one-launch sort

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

// VEC neighbouring elements as floats.
template <typename T, int VEC>
__device__ inline void em_load(const T *p, float (&o)[VEC]) {
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
__device__ inline void em_store(T *p, const float (&v)[VEC]) {
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

// ---------------------------------------------------------------- lookup
template <typename TE, typename TO, int VEC>
__global__ void __launch_bounds__(EM_THREADS) embed_kernel(const EmbedArgs a, int group, int rows, int *status) {
  griddep_launch();
  griddep_wait();
  const int sub = threadIdx.x / group, lane = threadIdx.x % group;
  const int64_t t0 = ((int64_t)blockIdx.x * (EM_THREADS / group) + sub) * rows;
  if (sub >= EM_THREADS / group) return;
  const TE *src[EM_ROWS];
#pragma unroll
  for (int r = 0; r < EM_ROWS; ++r) {
    src[r] = nullptr;
    if (r < rows && t0 + r < a.T) {
      const int64_t id = em_id(a, t0 + r);
      if (id >= 0 && id < a.V) src[r] = (const TE *)a.table + id * a.ld_table;
      else if (lane == 0) record_status(status, STATUS_BAD_TOKEN_ID);
    }
  }
  for (int i = lane * VEC; i < a.H; i += group * VEC) {
    float v[EM_ROWS][VEC];
#pragma unroll
    for (int r = 0; r < EM_ROWS; ++r) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[r][k] = 0.f;
      if (src[r]) em_load<TE, VEC>(src[r] + i, v[r]);
    }
#pragma unroll
    for (int r = 0; r < EM_ROWS; ++r)
      if (r < rows && t0 + r < a.T) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[r][k] *= a.scale;
        em_store<TO, VEC>((TO *)a.out + (t0 + r) * a.ld_out + i, v[r]);
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
embed_sort_kernel(const EmbedArgs a, int bits, int32_t *key1, int32_t *pos1, int32_t *key2, int32_t *pos2, int *status) {
  using namespace umma;
  extern __shared__ int32_t es_smem[];
  const int D = 1 << bits;
  int32_t *hist = es_smem, *total = hist + ES_WARPS * D, *wsum = total + D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  griddep_wait();
  griddep_launch();  // the zeroing may start: what came before has finished
  const int T = a.T;
  const int per_warp = (int)round_up(ceil_div(T, ES_CTAS * ES_WARPS), 32);
  const int begin = (rank * ES_WARPS + warp) * per_warp, end = min(begin + per_warp, T);
  int32_t *mine = hist + warp * D;
  for (int pass = 0; pass < 2; ++pass) {
    auto key_at = [&](int j) { return pass ? __ldcg(key1 + j) : em_key(a, j, status); };
    for (int d = threadIdx.x; d < ES_WARPS * D; d += ES_THREADS) hist[d] = 0;
    __syncthreads();
    for (int j = begin + lane; j < end; j += 32) atomicAdd(mine + ((key_at(j) >> (pass * bits)) & (D - 1)), 1);
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
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      const bool in = j < end;
      const int32_t key = in ? key_at(j) : -1;
      const int digit = in ? (key >> (pass * bits)) & (D - 1) : -1 - lane;
      const unsigned same = __match_any_sync(FULL_MASK, digit);
      const int ahead = __popc(same & lanemask_lt());
      int32_t base = 0;
      if (in) base = total[digit] + mine[digit];
      __syncwarp();
      if (in && ahead == 0) mine[digit] += __popc(same);
      __syncwarp();
      if (in) {
        (pass ? key2 : key1)[base + ahead] = key;
        (pass ? pos2 : pos1)[base + ahead] = pass ? __ldcg(pos1 + j) : j;
      }
    }
    if (pass == 0) {
      __threadfence();
      cluster_sync();
    }
  }
}

// The same by the permutation's kernels: low digits, then high digits.
__global__ void __launch_bounds__(256) embed_key_kernel(const EmbedArgs a, int32_t *key, int32_t *lo, int *status) {
  griddep_launch();
  griddep_wait();
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
// `beside`: runs beside the one-launch sort, which lets it start once it knows
// that what came before has finished, and waits for it at its end only, so
// that what follows waits for both.
__global__ void __launch_bounds__(512) embed_zero_kernel(float *p, int64_t n, int beside) {
  if (!beside) griddep_wait();
  const int64_t head = min(n, (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / 4), vecs = (n - head) / 4;
  float4 *v = (float4 *)(p + head);
  const int64_t i0 = blockIdx.x * 512ll + threadIdx.x, step = gridDim.x * 512ll;
  for (int64_t i = i0; i < vecs; i += step) __stcs(v + i, make_float4(0.f, 0.f, 0.f, 0.f));
  if (i0 < head) p[i0] = 0.f;
  if (i0 < n - head - 4 * vecs) p[head + 4 * vecs + i0] = 0.f;
  if (beside) griddep_wait();
}

// ---------------------------------------------------------------- sums
// Tiles of `tile` sorted positions; part: [tiles][2][H], a tile's sums of the
// token that was there before it (0) and of the one that goes on behind it (1).
template <typename TO, int VEC>
__global__ void __launch_bounds__(EM_THREADS)
embed_sum_kernel(const EmbedArgs a, int tile, int group, const int32_t *key, const int32_t *order, float *part) {
  constexpr int AHEAD = VEC == 1 ? 8 : 4;
  griddep_launch();
  griddep_wait();
  const int per_cta = EM_THREADS / group, sub = threadIdx.x / group;
  if (sub >= per_cta) return;
  const int64_t b = (int64_t)blockIdx.x * per_cta + sub;
  const int p0 = (int)min(b * tile, (int64_t)a.T), p1 = min(p0 + tile, a.T);
  if (p0 >= p1) return;
  const int first = key[p0];
  if (first >= a.V) return;
  const bool from_before = p0 > 0 && key[p0 - 1] == first;
  const int after = p1 < a.T ? key[p1] : a.V;
  const int i = (blockIdx.y * group + threadIdx.x % group) * VEC;
  if (i >= a.H) return;
  float s[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) s[k] = 0.f;
  int now = first;
  bool spans = from_before;
  auto flush = [&](bool goes_on) {
    if (spans || goes_on) {
      float *o = part + (b * 2 + (spans ? 0 : 1)) * a.H + i;
      if constexpr (VEC == 1) o[0] = s[0];
      else em_store<float, VEC>(o, s);
    } else {
      float *o = a.dtable + (int64_t)now * a.H + i;
      float v[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = 0.f;
      if (a.accumulate) em_load<float, VEC>(o, v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = a.accumulate ? fmaf(a.scale, s[k], v[k]) : a.scale * s[k];
      em_store<float, VEC>(o, v);
    }
  };
  for (int p = p0; p < p1; p += AHEAD) {
    float v[AHEAD][VEC];
    int k_at[AHEAD];
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      k_at[r] = p + r < p1 ? key[p + r] : a.V;
      if (k_at[r] < a.V) em_load<TO, VEC>((const TO *)a.dout + (int64_t)order[p + r] * a.ld_out + i, v[r]);
    }
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      if (p + r >= p1 || now >= a.V) break;
      if (k_at[r] != now) {
        flush(false);
        spans = false;
        now = k_at[r];
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] = 0.f;
        if (now >= a.V) break;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[k] += v[r][k];
    }
  }
  if (now < a.V) flush(after == now);
}

// A token that spans tiles: the tile that it starts in adds the partial rows
// up, in order.
__global__ void __launch_bounds__(EM_THREADS) embed_join_kernel(const EmbedArgs a, int tile, const int32_t *key,
                                                                const float *part) {
  griddep_launch();
  griddep_wait();
  const int64_t tiles = ceil_div(a.T, tile), b = blockIdx.x;
  const int p0 = (int)(b * tile), p1 = p0 + tile;
  if (p1 >= a.T) return;
  const int now = key[p1 - 1];
  if (now >= a.V || key[p1] != now) return;
  if (key[p0] == now && p0 > 0 && key[p0 - 1] == now) return;  // it started before
  // Tiles behind this one that it reaches.
  int64_t n = 0;
  for (;;) {
    const int64_t c = b + 1 + n + threadIdx.x;
    const int got = __syncthreads_count(c < tiles && key[c * tile] == now);
    n += got;
    if (got < EM_THREADS) break;
  }
  for (int i = blockIdx.y * EM_THREADS + threadIdx.x; i < a.H; i += gridDim.y * EM_THREADS) {
    float s = part[(b * 2 + 1) * a.H + i];
    const float *q = part + (b + 1) * 2 * (int64_t)a.H + i;
    int64_t c = 0;
    for (; c + 8 <= n; c += 8) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = q[(c + r) * 2 * a.H];
#pragma unroll
      for (int r = 0; r < 8; ++r) s += v[r];
    }
    for (; c < n; ++c) s += q[c * 2 * a.H];
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
  const int group = em_group(a.H, wide ? VEC : 1);
  // Four rows a group where there are enough of them to fill the SMs.
  const int rows = ceil_div(a.T, EM_THREADS / group) >= (int64_t)device_sms() * 2 * EM_ROWS ? EM_ROWS : 1;
  const dim3 grid((unsigned)ceil_div(a.T, (int64_t)(EM_THREADS / group) * rows)), block(EM_THREADS);
  if (wide) return launch_pdl(embed_kernel<TE, TO, VEC>, grid, block, 0, stream, a, group, rows, status);
  return launch_pdl(embed_kernel<TE, TO, 1>, grid, block, 0, stream, a, group, rows, status);
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
  int32_t *key, *order, *key1, *pos1, *lo, *second, *digits;
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
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a, bits, s.key1, s.pos1, s.key, s.order, status);
  }
  const int64_t T = a.T;
  const dim3 grid((unsigned)ceil_div(T, 256)), block(256);
  cudaError_t e = launch_pdl(embed_key_kernel, grid, block, 0, stream, a, s.key1, s.lo, status);
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
  const int vec = wide ? VEC : 1, group = em_group(a.H, vec), tile = em_tile(a.T);
  const int64_t tiles = ceil_div(a.T, tile);
  const dim3 grid((unsigned)ceil_div(tiles, EM_THREADS / group), (unsigned)ceil_div(a.H, group * vec));
  const int32_t *key = s.key, *order = s.order;
  cudaError_t e = wide ? launch_pdl(embed_sum_kernel<TO, VEC>, grid, dim3(EM_THREADS), 0, stream, a, tile, group, key, order, s.part)
                       : launch_pdl(embed_sum_kernel<TO, 1>, grid, dim3(EM_THREADS), 0, stream, a, tile, group, key, order, s.part);
  if (e != cudaSuccess || tiles < 2) return e;
  return launch_pdl(embed_join_kernel, dim3((unsigned)tiles, (unsigned)std::min<int64_t>(ceil_div(a.H, EM_THREADS), 64)), dim3(EM_THREADS), 0, stream, a,
                    tile, key, (const float *)s.part);
}

cudaError_t launch_embed_bwd(const EmbedArgs &a, void *scratch, int *status, cudaStream_t stream) {
  const int64_t n = (int64_t)a.V * a.H;
  if (a.T == 0) return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.dtable, 0, (size_t)n * sizeof(float), stream);
  size_t bytes;
  const EmbedScratch s = embed_carve(a, (char *)scratch, &bytes);
  cudaError_t e = embed_sort(a, s, status, stream);
  if (e == cudaSuccess && !a.accumulate) {
    const int64_t ctas = std::min<int64_t>(ceil_div(n, 512 * 16), (int64_t)device_sms() * 4);
    e = launch_pdl(embed_zero_kernel, dim3((unsigned)ctas), dim3(512), 0, stream, a.dtable, n, es_used(a) ? 1 : 0);
  }
  if (e != cudaSuccess) return e;
  return a.of32 ? embed_sum<float>(a, s, stream) : embed_sum<__nv_bfloat16>(a, s, stream);
}

}  // namespace moe

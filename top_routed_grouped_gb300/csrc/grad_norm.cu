// The global 2-norm of many tensors, and their scaling to a norm.
//
//   norm = sqrt(sum g^2)       out = in * min(1, max_norm / (norm + eps))
//
// Bound by memory: each gradient is read once for the norm and once more for
// the scaling, which starts at the end where the norm has stopped, so that
// what L2 still holds is read from there.  All tensors go in one launch: the
// table of them is a kernel argument (nothing to copy to the device, and a
// captured graph has it inside).  Tensors are cut into chunks of 8192
// elements; a CTA has a run of neighbouring chunks, finds the tensor of the first by
// bisection and goes on from there, forwards for the norm, backwards for the scaling.
//
// Squares are summed in FP32 over a chunk's 1024 elements of a warp (32 of a
// thread in four chains, then a tree), and only those sums in FP64: an SM adds
// two doubles a clock, and joining 256 threads' by a tree of them took as long
// as reading 40 MB.  Where a warp's sum is out of the range in which FP32 squares keep
// their bits (some |g| above 1e13, or all of them below 1e-12) its elements
// are read again and summed in FP64.  No atomics: each cluster leaves one partial
// sum, and all of them are added in one order.
//
// Measured: 6.5 GB of float clipped into bfloat16 in 2434 us (16.2 GB read and
// written: 6.65 TB/s, the copy rate); 600 MB of bfloat16 in 1500 tensors in 316 us
// (5.7 TB/s); the norm of 38 MB in 12 us from a graph, half of it launches.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"
#include "umma.cuh"

namespace moe {

constexpr int GN_THREADS = 256;
constexpr int GN_CTAS = 8;                   // CTAs a SM
constexpr int GN_CHUNK = 32 * GN_THREADS;    // elements
// CTAs of a cluster put their sums together on chip: every CTA of the scaling
// adds all partial sums up.
constexpr int GN_CLUSTER = 8;

// CAP tensors: 28 bytes each, of the 32 KB that a kernel's arguments may take.
template <int CAP>
struct GradTable {
  const void *in[CAP];
  void *out[CAP];
  int64_t size[CAP];    // elements
  int first[CAP + 1];   // chunks before this tensor's
  uint32_t f32[CAP / 32], of32[CAP / 32];
  int n;
};
constexpr int GN_SMALL = 64, GN_LARGE = 1024;
static_assert(sizeof(GradTable<GN_LARGE>) <= 32000, "a kernel's arguments");

// The tensor of a chunk: the last one whose first chunk is not behind it.
template <int CAP>
__device__ inline int tensor_of(const GradTable<CAP> &t, int chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Elements before the first 16-byte boundary.
template <typename E>
__device__ inline int head_of(const E *p, int64_t n) {
  const int h = (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(E));
  return n < h ? (int)n : h;
}

template <typename T>
__device__ inline T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

// The sum of the squares of this warp's elements of chunk c of a tensor: the
// head (chunk 0), units of 16 bytes, the tail (the last chunk).
template <typename E>
__device__ inline double chunk_squares(const E *p, int64_t n, int c, int nchunks) {
  constexpr int N = Vec16<E>::N;
  const int head = head_of(p, n);
  const int64_t units = (n - head) / N, per = GN_CHUNK / N;
  const int64_t u0 = c * per, u1 = c + 1 == nchunks ? units : min(units, u0 + per);
  const uint4 *v = (const uint4 *)(p + head);
  const int tail = (int)(n - head - units * N);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t any = 0;  // a bit that is not a sign
  auto unit = [&](const uint4 &w, float &a, float &b) {
    float x[N];
    Vec16<E>::unpack(w, x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      a = fmaf(x[i], x[i], a);
      b = fmaf(x[i + 1], x[i + 1], b);
    }
    any |= w.x | w.y | w.z | w.w;
  };
  int64_t u = u0 + threadIdx.x;
  constexpr int B = 32 / N;  // units of a thread: all of them in flight
  if (u0 + per <= u1) {
    uint4 w[B];
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = v[u + i * GN_THREADS];
#pragma unroll
    for (int i = 0; i < B; ++i) unit(w[i], s[2 * i & 2], s[(2 * i & 2) + 1]);
  } else {
    for (; u < u1; u += GN_THREADS) unit(v[u], s[0], s[1]);
  }
  // At most one element of the head and one of the tail a thread.
  float edge[2] = {0.f, 0.f};
  if (c == 0 && (int)threadIdx.x < head) edge[0] = Elem<E>::load(p + threadIdx.x);
  if (c + 1 == nchunks && (int)threadIdx.x < tail) edge[1] = Elem<E>::load(p + head + units * N + threadIdx.x);
  s[2] = fmaf(edge[0], edge[0], s[2]);
  s[3] = fmaf(edge[1], edge[1], s[3]);
  any |= __float_as_uint(edge[0]) | __float_as_uint(edge[1]);
  const float sum = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
  const uint32_t signs = sizeof(E) == 2 ? 0x7fff7fffu : 0x7fffffffu;
  if (sum < 1e30f && (sum > 1e-24f || !__any_sync(FULL_MASK, (any & signs) != 0))) return sum;
  double d = (double)edge[0] * edge[0] + (double)edge[1] * edge[1];
  for (u = u0 + threadIdx.x; u < u1; u += GN_THREADS) {
    float x[N];
    Vec16<E>::unpack(v[u], x);
#pragma unroll
    for (int i = 0; i < N; ++i) d += (double)x[i] * x[i];
  }
  return warp_sum(d);
}

// The run of chunks of this CTA.
__device__ inline void run_of(int total, int &c0, int &c1) {
  c0 = (int)((int64_t)total * blockIdx.x / gridDim.x);
  c1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
}

template <int CAP>
__global__ void __launch_bounds__(GN_THREADS)
grad_norm_kernel(const __grid_constant__ GradTable<CAP> t, double *part) {
  umma::cluster_meet_arrive();
  griddep_launch();
  int c0, c1;
  run_of(t.first[t.n], c0, c1);
  int i = c1 > c0 ? tensor_of(t, c0) : 0;
  griddep_wait();
  double sum = 0;
  for (int c = c0; c < c1; ++c) {
    if (c == t.first[i + 1]) ++i;  // (no tensor of the table is empty)
    const int first = t.first[i], k = t.first[i + 1] - first;
    if (t.f32[i >> 5] >> (i & 31) & 1) sum += chunk_squares((const float *)t.in[i], t.size[i], c - first, k);
    else sum += chunk_squares((const __nv_bfloat16 *)t.in[i], t.size[i], c - first, k);
  }
  // All warps of the cluster to its first CTA, where one thread adds them in order.
  constexpr int WARPS = GN_THREADS / 32;
  __shared__ double of_cluster[GN_CLUSTER * WARPS];
  const uint32_t rank = umma::cluster_ctarank();
  umma::cluster_meet_wait();  // the first CTA runs: its shared memory is there to be written (behind the reads at no cost)
  if ((threadIdx.x & 31) == 0)
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                     umma::mapa_shared(&of_cluster[rank * WARPS + (threadIdx.x >> 5)], 0)),
                 "d"(sum)
                 : "memory");
  umma::cluster_sync();
  if (rank == 0 && threadIdx.x < 32) {
    double s = 0;
#pragma unroll
    for (int i = 0; i < GN_CLUSTER * WARPS / 32; ++i) s += of_cluster[i * 32 + threadIdx.x];
    s = warp_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x / GN_CLUSTER] = s;
  }
}

// All partial sums, in one order, by the CTA's first warp.
__device__ inline float norm_of(const double *part, int n) {
  __shared__ float norm;
  if (threadIdx.x < 32) {
    double s = 0;
    for (int i = threadIdx.x; i < n; i += 32) s += part[i];
    s = warp_sum(s);
    if (threadIdx.x == 0) norm = (float)sqrt(s);
  }
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(32) grad_norm_finish_kernel(const double *part, int n, float *norm) {
  griddep_launch();
  griddep_wait();
  const float r = norm_of(part, n);
  if (threadIdx.x == 0) *norm = r;
}

template <typename I, typename O>
__device__ inline void chunk_scale(const I *in, O *out, int64_t n, int c, int nchunks, float f) {
  // Groups of eight elements that start on a 16-byte boundary of the output.
  const int head = head_of(out, n);
  const int64_t groups = (n - head) / 8, per = GN_CHUNK / 8;
  const int64_t g0 = c * per, g1 = c + 1 == nchunks ? groups : min(groups, g0 + per);
  const int tail = (int)(n - head - groups * 8);
  const I *pi = in + head;
  O *po = out + head;
  constexpr int NI = Vec16<I>::N, NO = Vec16<O>::N;
  const bool wide = ((uintptr_t)pi & 15) == 0;
  if (wide && g0 + per <= g1) {  // a whole chunk: all of a thread's groups in flight
    const int64_t g = g0 + threadIdx.x;
    uint4 w[4][8 / NI];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8 / NI; ++i) w[j][i] = *((const uint4 *)(pi + (g + j * GN_THREADS) * 8) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8 / NI; ++i) Vec16<I>::unpack(w[j][i], *(float(*)[NI])&x[i * NI]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
#pragma unroll
      for (int i = 0; i < 8 / NO; ++i) Vec16<O>::store(po + (g + j * GN_THREADS) * 8 + i * NO, *(float(*)[NO])&x[i * NO]);
    }
  } else {
    for (int64_t g = g0 + threadIdx.x; g < g1; g += GN_THREADS) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = Elem<I>::load(pi + g * 8 + i) * f;
#pragma unroll
      for (int i = 0; i < 8 / NO; ++i) Vec16<O>::store(po + g * 8 + i * NO, *(float(*)[NO])&x[i * NO]);
    }
  }
  if (c == 0 && (int)threadIdx.x < head)
    out[threadIdx.x] = Elem<O>::from_f32(Elem<I>::load(in + threadIdx.x) * f);
  if (c + 1 == nchunks && (int)threadIdx.x < tail) {
    const int64_t at = groups * 8 + threadIdx.x;
    po[at] = Elem<O>::from_f32(Elem<I>::load(pi + at) * f);
  }
}

// part: the partial sums (the clip; CTA 0 writes the norm), or NULL: the norm is given.
template <int CAP>
__global__ void __launch_bounds__(GN_THREADS)
grad_scale_kernel(const __grid_constant__ GradTable<CAP> t, const double *part, int nparts, float max_norm, float eps,
                  float *norm) {
  griddep_launch();
  int c0, c1;
  run_of(t.first[t.n], c0, c1);
  int i = c1 > c0 ? tensor_of(t, c1 - 1) : 0;
  griddep_wait();
  float r;
  if (part) {
    r = norm_of(part, nparts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
  } else {
    r = *norm;
  }
  float f = max_norm / (r + eps);
  if (f > 1.f) f = 1.f;  // (NaN stays)
  for (int c = c1 - 1; c >= c0; --c) {
    if (c < t.first[i]) --i;
    if (f == 1.f && t.in[i] == t.out[i]) continue;
    const int first = t.first[i], k = t.first[i + 1] - first;
    const int64_t n = t.size[i];
    const bool a = t.f32[i >> 5] >> (i & 31) & 1, b = t.of32[i >> 5] >> (i & 31) & 1;
    if (a && b) chunk_scale((const float *)t.in[i], (float *)t.out[i], n, c - first, k, f);
    else if (a) chunk_scale((const float *)t.in[i], (__nv_bfloat16 *)t.out[i], n, c - first, k, f);
    else if (b) chunk_scale((const __nv_bfloat16 *)t.in[i], (float *)t.out[i], n, c - first, k, f);
    else chunk_scale((const __nv_bfloat16 *)t.in[i], (__nv_bfloat16 *)t.out[i], n, c - first, k, f);
  }
}

// ------------------------------------------------------------------ host side
static int launches(const GradList &a) { return std::max(1, (int)ceil_div(a.n, GN_LARGE)); }

// CTAs of a launch at most.
static int most_ctas() { return std::max(1, device_sms()) * GN_CTAS; }

size_t grad_scratch_bytes(const GradList &a) { return (size_t)launches(a) * (most_ctas() / GN_CLUSTER) * sizeof(double); }

// Tensors [i0, i1) of the list; the number of chunks.
template <int CAP>
static int fill(GradTable<CAP> &t, const GradList &a, int i0, int i1, bool out) {
  t.n = 0;
  int chunks = 0;
  for (int i = 0; i < CAP / 32; ++i) t.f32[i] = t.of32[i] = 0;
  for (int i = i0; i < i1; ++i) {
    if (a.numel[i] == 0) continue;
    const int k = t.n++;
    t.in[k] = a.in[i];
    t.out[k] = out ? a.out[i] : nullptr;
    t.size[k] = a.numel[i];
    t.first[k] = chunks;
    chunks += (int)ceil_div(a.numel[i], GN_CHUNK);
    if (a.dtype[i] == 0) t.f32[k >> 5] |= 1u << (k & 31);
    if (out && a.odtype[i] == 0) t.of32[k >> 5] |= 1u << (k & 31);
  }
  t.first[t.n] = chunks;
  return chunks;
}

template <int CAP>
static cudaError_t run(const GradList &a, int mode, double *part, cudaStream_t stream) {
  const int most = most_ctas();
  const int nl = (int)ceil_div(a.n, CAP);
  GradTable<CAP> t;
  cudaError_t e;
  int parts = 0;
  if (mode & GRAD_NORM) {
    for (int l = 0; l < nl; ++l) {
      const int chunks = fill(t, a, l * CAP, std::min(a.n, (l + 1) * CAP), false);
      if (!chunks) continue;
      const int grid = (int)round_up(std::min(chunks, most), GN_CLUSTER);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(grid);
      cfg.blockDim = dim3(GN_THREADS);
      cfg.stream = stream;
      cudaLaunchAttribute at[2];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = GN_CLUSTER;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[1].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 2;
      if ((e = cudaLaunchKernelEx(&cfg, grad_norm_kernel<CAP>, t, part + parts)) != cudaSuccess) return e;
      parts += grid / GN_CLUSTER;
    }
  }
  if (mode == GRAD_NORM)
    return launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(32), 0, stream, (const double *)part, parts, a.norm);
  const double *p = mode & GRAD_NORM ? part : nullptr;
  bool any = false;
  for (int l = nl - 1; l >= 0; --l) {
    const int chunks = fill(t, a, l * CAP, std::min(a.n, (l + 1) * CAP), true);
    if (!chunks && (l || any)) continue;  // (of an empty list the norm is still written)
    any = true;
    e = launch_pdl(grad_scale_kernel<CAP>, dim3(std::max(1, std::min(chunks, most))), dim3(GN_THREADS), 0, stream, t, p,
                   parts, a.max_norm, a.eps, a.norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_grads(const GradList &a, int mode, void *scratch, cudaStream_t stream) {
  if (a.n == 0 && mode != GRAD_SCALE)
    return launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(32), 0, stream, (const double *)scratch, 0, a.norm);
  return a.n <= GN_SMALL ? run<GN_SMALL>(a, mode, (double *)scratch, stream)
                         : run<GN_LARGE>(a, mode, (double *)scratch, stream);
}

}  // namespace moe

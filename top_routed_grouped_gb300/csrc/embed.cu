// Token embedding with a scale, and its gradient by sorted tokens (contracts
// with moe_embed in moe.h).
//
// Gradient: the tokens are sorted by a stable counting sort in two digits of
// ten bits (low, then high), so that the rows of one token stand in ascending
// t; each row of the table then sums its run.  Tokens left out (outside the
// table, or the padding token) sort behind the table as token V.
#include "common.cuh"
#include "kernels.h"
#include "tc_host.h"

namespace moe {

constexpr int EM_THREADS = 256, EM_DIGIT = 1024;

__device__ inline int64_t em_id(const EmbedArgs &a, int64_t t) {
  return a.ids64 ? ((const int64_t *)a.ids)[t] : (int64_t)((const int32_t *)a.ids)[t];
}

template <typename TE, typename TO>
__global__ void __launch_bounds__(EM_THREADS) embed_kernel(const EmbedArgs a, int *status) {
  griddep_launch();
  griddep_wait();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t id = em_id(a, t);
    const bool ok = id >= 0 && id < a.V;
    if (!ok && threadIdx.x == 0) record_status(status, STATUS_BAD_TOKEN_ID);
    for (int i = threadIdx.x; i < a.H; i += EM_THREADS) {
      const float v = ok ? a.scale * Elem<TE>::load((const TE *)a.table + id * a.ld_table + i) : 0.f;
      ((TO *)a.out)[t * a.ld_out + i] = Elem<TO>::from_f32(v);
    }
  }
}

// key[t] = the token, V where it is left out; lo = its low digit.
__global__ void __launch_bounds__(256) embed_key_kernel(const EmbedArgs a, int32_t *key, int32_t *lo, int *status) {
  griddep_launch();
  griddep_wait();
  for (int64_t t = blockIdx.x * 256ll + threadIdx.x; t < a.T; t += gridDim.x * 256ll) {
    const int64_t id = em_id(a, t);
    const bool ok = id >= 0 && id < a.V;
    if (!ok) record_status(status, STATUS_BAD_TOKEN_ID);
    const int32_t k = ok && id != a.padding_id ? (int32_t)id : a.V;
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

// order[j] = t of sorted position j, start[v] = first position of token v.
__global__ void __launch_bounds__(256) embed_order_kernel(int64_t T, int V, const int32_t *key, const int32_t *first,
                                                          const int32_t *second, int32_t *order, int32_t *start) {
  griddep_launch();
  griddep_wait();
  for (int64_t j = blockIdx.x * 256ll + threadIdx.x; j <= T; j += gridDim.x * 256ll) {
    const int t = j < T ? first[second[j]] : 0;
    const int k = j < T ? key[t] : V;
    const int before = j > 0 ? key[first[second[j - 1]]] : -1;
    if (j < T) order[j] = t;
    for (int v = before + 1; v <= k; ++v) start[v] = (int32_t)j;
  }
}

template <typename TO>
__global__ void __launch_bounds__(EM_THREADS) embed_sum_kernel(const EmbedArgs a, const int32_t *order,
                                                               const int32_t *start) {
  griddep_launch();
  griddep_wait();
  for (int64_t v = blockIdx.x; v < a.V; v += gridDim.x) {
    const int32_t lo = start[v], hi = start[v + 1];
    if (a.accumulate && lo == hi) continue;
    for (int i = threadIdx.x; i < a.H; i += EM_THREADS) {
      float s = 0.f;
      for (int32_t j = lo; j < hi; ++j) s += Elem<TO>::load((const TO *)a.dout + (int64_t)order[j] * a.ld_out + i);
      float *o = a.dtable + v * a.H + i;
      *o = a.accumulate ? fmaf(a.scale, s, *o) : a.scale * s;
    }
  }
}

cudaError_t launch_embed(const EmbedArgs &a, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const dim3 grid((unsigned)a.T);
  if (a.f32) return launch_pdl(embed_kernel<float, float>, grid, dim3(EM_THREADS), 0, stream, a, status);
  if (a.of32) return launch_pdl(embed_kernel<__nv_bfloat16, float>, grid, dim3(EM_THREADS), 0, stream, a, status);
  return launch_pdl(embed_kernel<__nv_bfloat16, __nv_bfloat16>, grid, dim3(EM_THREADS), 0, stream, a, status);
}

struct EmbedScratch {
  int32_t *key, *digit, *first, *second, *pos, *order, *start, *digits;
  void *sort;
};
static EmbedScratch embed_carve(const EmbedArgs &a, char *base, size_t *bytes) {
  size_t off = 0;
  auto take = [&](size_t n) {
    char *p = base + off;
    off += (n + 255) / 256 * 256;
    return p;
  };
  EmbedScratch s;
  const size_t t = (size_t)a.T * 4;
  s.key = (int32_t *)take(t);
  s.digit = (int32_t *)take(t);
  s.first = (int32_t *)take(t);
  s.second = (int32_t *)take(t);
  s.pos = (int32_t *)take(t);
  s.order = (int32_t *)take(t);
  s.start = (int32_t *)take(((size_t)a.V + 2) * 4);
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

cudaError_t launch_embed_bwd(const EmbedArgs &a, void *scratch, int *status, cudaStream_t stream) {
  if (a.T == 0)
    return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.dtable, 0, (size_t)a.V * a.H * sizeof(float), stream);
  size_t n;
  const EmbedScratch s = embed_carve(a, (char *)scratch, &n);
  const dim3 grid((unsigned)ceil_div((int64_t)a.T + 1, 256)), block(256);
  cudaError_t e = launch_pdl(embed_key_kernel, grid, block, 0, stream, a, s.key, s.digit, status);
  if (e == cudaSuccess) e = launch_permute(a.T, EM_DIGIT, s.digit, s.digits, s.first, s.pos, s.sort, status, stream);
  if (e == cudaSuccess)
    e = launch_pdl(embed_high_kernel, grid, block, 0, stream, (int64_t)a.T, (const int32_t *)s.key, (const int32_t *)s.first, s.digit);
  if (e == cudaSuccess) e = launch_permute(a.T, EM_DIGIT, s.digit, s.digits, s.second, s.pos, s.sort, status, stream);
  if (e == cudaSuccess)
    e = launch_pdl(embed_order_kernel, grid, block, 0, stream, (int64_t)a.T, a.V, (const int32_t *)s.key, (const int32_t *)s.first,
                   (const int32_t *)s.second, s.order, s.start);
  if (e != cudaSuccess) return e;
  const dim3 rows((unsigned)a.V);
  if (a.of32) return launch_pdl(embed_sum_kernel<float>, rows, dim3(EM_THREADS), 0, stream, a, (const int32_t *)s.order, (const int32_t *)s.start);
  return launch_pdl(embed_sum_kernel<__nv_bfloat16>, rows, dim3(EM_THREADS), 0, stream, a, (const int32_t *)s.order, (const int32_t *)s.start);
}

}  // namespace moe

// The join between two blocks: launches, and the sums over rows of the
// weights' gradients (the kernels over rows are in block_norm.cuh; one type of
// rows is compiled here, the others beside it).
#include "block_norm.cuh"

namespace moe {

extern template cudaError_t bn_dispatch<float, float>(const BnLaunch &);
extern template cudaError_t bn_dispatch<__nv_bfloat16, float>(const BnLaunch &);

// out[i] = sum over the CTAs (`groups`) of part[.][i], in a fixed order: 32
// threads of a column take every 32nd, then a tree.
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

static cudaError_t bn_any(const BnLaunch &l) {
  if (l.a.f32) return bn_dispatch<float, float>(l);
  if (l.a.rf32) return bn_dispatch<__nv_bfloat16, float>(l);
  return bn_dispatch<__nv_bfloat16, __nv_bfloat16>(l);
}

cudaError_t launch_block_norm(const NormArgs &a, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return bn_any({a, false, nullptr, status, stream, nullptr});
}

size_t block_norm_scratch_bytes(const NormArgs &a) {
  return a.T == 0 ? 0 : (size_t)3 * bn_most_ctas(a) * a.H * sizeof(float);
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
  cudaError_t e = bn_any({a, true, (float *)scratch, status, stream, &groups});
  if (e != cudaSuccess || (!a.dw_pre && !a.dw_post && !dg)) return e;
  return launch_pdl(block_norm_join_kernel, dim3((unsigned)ceil_div(a.H, 32), 3), dim3(32, 32), 0, stream,
                    (const float *)scratch, (int64_t)groups, a.H, a.dw_pre, a.dw_post, dg);
}

}  // namespace moe

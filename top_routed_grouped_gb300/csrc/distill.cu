// Distillation from a teacher's top logits, bfloat16 logits (the kernels are
// in distill.cuh; the float ones are compiled beside them).
#include "distill.cuh"

namespace moe {

extern template cudaError_t distill_launch<float>(const DistillArgs &, int, int *, cudaStream_t);

cudaError_t launch_distill(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.f32 ? distill_launch<float>(a, mode, status, stream) : distill_launch<__nv_bfloat16>(a, mode, status, stream);
}

}  // namespace moe

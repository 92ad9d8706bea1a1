// Distillation from a teacher's top logits: choice of the kernels (they are in
// distill.cuh; those of one type and alignment are compiled here, the others
// beside it).
#include "distill.cuh"

namespace moe {

extern template cudaError_t ds_mode<float, true>(const DistillArgs &, int, int *, cudaStream_t);
extern template cudaError_t ds_mode<float, false>(const DistillArgs &, int, int *, cudaStream_t);
extern template cudaError_t ds_mode<__nv_bfloat16, false>(const DistillArgs &, int, int *, cudaStream_t);

template <typename T>
static cudaError_t distill_type(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  constexpr int N = 16 / (int)sizeof(T);
  bool aligned = (uintptr_t)a.logits % 16 == 0 && a.ld_logits % N == 0;
  if (mode & DISTILL_GRAD) aligned = aligned && (uintptr_t)a.dlogits % 16 == 0 && a.ld_dlogits % N == 0;
  return aligned ? ds_mode<T, true>(a, mode, status, stream) : ds_mode<T, false>(a, mode, status, stream);
}

cudaError_t launch_distill(const DistillArgs &a, int mode, int *status, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.f32 ? distill_type<float>(a, mode, status, stream) : distill_type<__nv_bfloat16>(a, mode, status, stream);
}

}  // namespace moe

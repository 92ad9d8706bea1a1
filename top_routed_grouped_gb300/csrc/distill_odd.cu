// Distillation from a teacher's top logits, bfloat16 rows between 16-byte boundaries.
#include "distill.cuh"

namespace moe {

template cudaError_t ds_mode<__nv_bfloat16, false>(const DistillArgs &, int, int *, cudaStream_t);

}  // namespace moe

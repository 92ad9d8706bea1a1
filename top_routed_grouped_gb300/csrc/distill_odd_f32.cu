// Distillation from a teacher's top logits, float rows between 16-byte boundaries.
#include "distill.cuh"

namespace moe {

template cudaError_t ds_mode<float, false>(const DistillArgs &, int, int *, cudaStream_t);

}  // namespace moe

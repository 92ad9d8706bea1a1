// Distillation from a teacher's top logits, float logits.
#include "distill.cuh"

namespace moe {

template cudaError_t ds_mode<float, true>(const DistillArgs &, int, int *, cudaStream_t);

}  // namespace moe

// Distillation from a teacher's top logits, float logits.
#include "distill.cuh"

namespace moe {

template cudaError_t distill_launch<float>(const DistillArgs &, int, int *, cudaStream_t);

}  // namespace moe

// The join between two blocks, float rows.
#include "block_norm.cuh"

namespace moe {

template cudaError_t bn_dispatch<float, float>(const BnLaunch &);

}  // namespace moe

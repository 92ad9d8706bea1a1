// The join between two blocks, bfloat16 rows beside a float residual.
#include "block_norm.cuh"

namespace moe {

template cudaError_t bn_dispatch<__nv_bfloat16, float>(const BnLaunch &);

}  // namespace moe

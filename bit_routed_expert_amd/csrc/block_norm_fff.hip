// Instantiation of the block norms: x fp32, y fp32, u fp32.
#include "block_norm_impl.hpp"

namespace strata {
template hipError_t block_norm_launch<float, float, float>(const NormArgs &, bool, hipStream_t);
}  // namespace strata

// Instantiation of the block norms: x bf16, y bf16, u bf16.
#include "block_norm_impl.hpp"

namespace strata {
template hipError_t block_norm_launch<uint16_t, uint16_t, uint16_t>(const NormArgs &, bool, hipStream_t);
}  // namespace strata

// Instantiation of the block norms for rows whose length is no multiple of 8.
#include "block_norm_impl.hpp"

namespace strata {
template hipError_t block_norm_launch_any<2>(const NormArgs &, bool, hipStream_t);
template hipError_t block_norm_launch_any<1>(const NormArgs &, bool, hipStream_t);
}  // namespace strata

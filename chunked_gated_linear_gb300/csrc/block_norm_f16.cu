// block_norm_f16.cu -- block_norm for rows of __half and a residual stream of __half.
#include "block_norm.cuh"

namespace gcl {
namespace blk {
GCL_BLOCK_NORM(__half, __half)
}  // namespace blk
}  // namespace gcl

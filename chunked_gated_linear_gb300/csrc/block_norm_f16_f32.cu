// block_norm_f16_f32.cu -- block_norm for rows of __half and a residual stream of float.
#include "block_norm.cuh"

namespace gcl {
namespace blk {
GCL_BLOCK_NORM(__half, float)
}  // namespace blk
}  // namespace gcl

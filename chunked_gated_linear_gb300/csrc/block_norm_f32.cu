// block_norm_f32.cu -- block_norm for rows of float and a residual stream of float.
#include "block_norm.cuh"

namespace gcl {
namespace blk {
GCL_BLOCK_NORM(float, float)
}  // namespace blk
}  // namespace gcl

// block_norm_bf16_f32.cu -- block_norm for rows of __nv_bfloat16 and a residual stream of float.
#include "block_norm.cuh"

namespace gcl {
namespace blk {
GCL_BLOCK_NORM(__nv_bfloat16, float)
}  // namespace blk
}  // namespace gcl

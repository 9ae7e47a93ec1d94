// block_norm_bf16.cu -- block_norm for rows of __nv_bfloat16 and a residual stream of __nv_bfloat16.
#include "block_norm.cuh"

namespace gcl {
namespace blk {
GCL_BLOCK_NORM(__nv_bfloat16, __nv_bfloat16)
}  // namespace blk
}  // namespace gcl

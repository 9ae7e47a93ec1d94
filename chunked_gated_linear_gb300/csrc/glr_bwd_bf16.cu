// glr_bwd_bf16.cu -- gated linear recurrence, backward, for rows of __nv_bfloat16.
#include "glr_bwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_bwd<__nv_bfloat16>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

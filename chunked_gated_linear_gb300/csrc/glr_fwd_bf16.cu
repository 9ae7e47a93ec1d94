// glr_fwd_bf16.cu -- gated linear recurrence, forward, for rows of __nv_bfloat16.
#include "glr_fwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_fwd<__nv_bfloat16>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

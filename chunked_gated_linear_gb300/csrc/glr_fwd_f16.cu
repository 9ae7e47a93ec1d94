// glr_fwd_f16.cu -- gated linear recurrence, forward, for rows of __half.
#include "glr_fwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_fwd<__half>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

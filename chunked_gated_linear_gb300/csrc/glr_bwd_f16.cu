// glr_bwd_f16.cu -- gated linear recurrence, backward, for rows of __half.
#include "glr_bwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_bwd<__half>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

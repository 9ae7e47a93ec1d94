// glr_fwd_f32.cu -- gated linear recurrence, forward, for rows of float.
#include "glr_fwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_fwd<float>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

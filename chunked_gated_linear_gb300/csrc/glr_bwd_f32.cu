// glr_bwd_f32.cu -- gated linear recurrence, backward, for rows of float.
#include "glr_bwd.cuh"

namespace gcl {
namespace glr {
template cudaError_t launch_bwd<float>(const Params &, cudaStream_t);
}  // namespace glr
}  // namespace gcl

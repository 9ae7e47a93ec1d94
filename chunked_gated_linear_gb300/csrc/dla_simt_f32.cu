// dla_simt_f32.cu -- instantiates the CUDA-core engine of decayed linear attention for f32 rows.
#include "dla_simt.cuh"

namespace gcl {
namespace dla {
template cudaError_t launch_simt_t<float>(const Params &, bool, int, const int *, cudaStream_t);
}
}  // namespace gcl

// dla_simt_f16.cu -- instantiates the CUDA-core engine of decayed linear attention for f16 rows.
#include "dla_simt.cuh"

namespace gcl {
namespace dla {
template cudaError_t launch_simt_t<__half>(const Params &, bool, int, const int *, cudaStream_t);
}
}  // namespace gcl

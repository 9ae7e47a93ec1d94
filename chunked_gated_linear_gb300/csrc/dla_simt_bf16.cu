// dla_simt_bf16.cu -- instantiates the CUDA-core engine of decayed linear attention for bf16 rows.
#include "dla_simt.cuh"

namespace gcl {
namespace dla {
template cudaError_t launch_simt_t<__nv_bfloat16>(const Params &, bool, int, const int *, cudaStream_t);
}
}  // namespace gcl

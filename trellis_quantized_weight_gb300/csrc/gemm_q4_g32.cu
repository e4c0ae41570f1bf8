// Products with 4-bit weights, groups of 32: the kernels of gemm_q4_mma.cuh.
#include "gemm_q4_mma.cuh"

namespace trellis {

template cudaError_t launch_q4_mma<32>(const Q4Args&, const DeviceInfo&, cudaStream_t);

}  // namespace trellis

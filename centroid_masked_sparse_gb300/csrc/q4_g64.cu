// 4-bit products with groups of 64 columns.
#include "q4_kernel.cuh"

namespace mtp {

template cudaError_t launch_q4_group<64>(const Q4Params &, cudaStream_t);

}  // namespace mtp

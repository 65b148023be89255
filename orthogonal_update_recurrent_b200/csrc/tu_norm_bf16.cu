// tu_norm_bf16.cu -- the block norms' kernels for calls of this type.
#include "common.cuh"
#include "norm_launch.cuh"

namespace lattice {

template lattice_status norm::launch_norm<__nv_bfloat16>(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);

cudaError_t status_norm_bf16(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

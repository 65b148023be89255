// tu_norm_f16.cu -- the block norms' kernels for calls of this type.
#include "common.cuh"
#include "norm_launch.cuh"

namespace lattice {

template lattice_status norm::launch_norm<__half>(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);

cudaError_t status_norm_f16(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

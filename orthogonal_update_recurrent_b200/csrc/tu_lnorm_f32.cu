// tu_lnorm_f32.cu -- the layer norm's kernels for calls of this type.
#include "common.cuh"
#include "lnorm_launch.cuh"

namespace lattice {

template lattice_status norm::launch_layer<float>(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);

int layer_parts(long long N, int D) { return norm::parts(N, D, false); }

cudaError_t status_lnorm_f32(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

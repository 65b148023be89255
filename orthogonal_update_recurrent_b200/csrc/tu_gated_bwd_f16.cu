// tu_gated_bwd_f16.cu -- the gated recurrence's backward kernels for x of this type.
#include "common.cuh"
#include "gated_bwd_launch.cuh"

namespace lattice {

template lattice_status gated::launch_bwd<__half>(GatedArgs a, int form, bool vec, cudaStream_t st);

cudaError_t status_gated_bwd_f16(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

// tu_gated_fwd_f16.cu -- the gated recurrence's forward and single-token kernels for x of this type.
#include "common.cuh"
#include "gated_fwd_launch.cuh"

namespace lattice {

template lattice_status gated::launch_fwd<__half>(GatedArgs a, int form, bool vec, cudaStream_t st);
template lattice_status gated::launch_step<__half>(const GatedArgs& a, int form, bool vec, cudaStream_t st);

cudaError_t status_gated_fwd_f16(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

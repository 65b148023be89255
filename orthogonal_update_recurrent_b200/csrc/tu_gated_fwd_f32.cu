// tu_gated_fwd_f32.cu -- the gated recurrence's forward and single-token kernels for x of this type.
#include "common.cuh"
#include "gated_fwd_launch.cuh"

namespace lattice {

template lattice_status gated::launch_fwd<float>(GatedArgs a, int form, bool vec, cudaStream_t st);
template lattice_status gated::launch_step<float>(const GatedArgs& a, int form, bool vec, cudaStream_t st);

cudaError_t status_gated_fwd_f32(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

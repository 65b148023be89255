// tu_gated_fwd_bf16.cu -- the gated recurrence's forward and single-token kernels for x of this type.
#include "common.cuh"
#include "gated_fwd_launch.cuh"

namespace lattice {

template lattice_status gated::launch_fwd<__nv_bfloat16>(GatedArgs a, int form, bool vec, cudaStream_t st);
template lattice_status gated::launch_step<__nv_bfloat16>(const GatedArgs& a, int form, bool vec, cudaStream_t st);

cudaError_t status_gated_fwd_bf16(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

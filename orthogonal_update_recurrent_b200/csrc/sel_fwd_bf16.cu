// sel_fwd_bf16.cu -- the selective scan's forward and single-token kernels for x of this type.
#include "selective_launch.cuh"

namespace lattice {

template lattice_status selective::launch_fwd<__nv_bfloat16>(const SelArgs& a, int S, int W, cudaStream_t st);
template lattice_status selective::launch_step<__nv_bfloat16>(const SelArgs& a, cudaStream_t st);

}  // namespace lattice

// sel_bwd_bf16.cu -- the selective scan's backward kernels for x of this type.
#include "selective_launch.cuh"

namespace lattice {

template lattice_status selective::launch_bwd<__nv_bfloat16>(const SelArgs& a, int W, cudaStream_t st);

}  // namespace lattice

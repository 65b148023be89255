// sel_bwd_f32.cu -- the selective scan's backward kernels for x of this type.
#include "selective_launch.cuh"

namespace lattice {

template lattice_status selective::launch_bwd<float>(const SelArgs& a, int W, cudaStream_t st);

}  // namespace lattice

// conv_f32.cu -- the short convolution's kernels for x of this type.
#include "conv_launch.cuh"

namespace lattice {

template lattice_status conv::launch<float>(const ConvArgs& a, int what, int V, cudaStream_t st);

}  // namespace lattice

// tu_norm_f32.cu -- the block norms' kernels for calls of this type.
#include "common.cuh"
#include "norm_launch.cuh"

namespace lattice {

template lattice_status norm::launch_norm<float>(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);

int norm_parts(long long N, int D) { return norm::parts(N, D, true); }

lattice_status launch_norm_dw(const NormArgs& a, int groups, float* dw_post, float* dw_pre, cudaStream_t st) {
    norm::norm_dw_kernel<32><<<(unsigned)((2 * a.D + 31) / 32), 1024, 0, st>>>(a.parts, groups, a.D, a.scale,
                                                                             dw_post, dw_pre);
    return launch_status();
}

cudaError_t status_norm_f32(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

// gated_launch.cuh -- what the launches of the gated recurrence's two directions share.
#pragma once
#include <type_traits>

#include "gated.cuh"
#include "launch.h"

namespace lattice {
namespace gated {

// CTAs per cluster: the most, by doubling, with which the grid is still resident at once
// (`resident` CTAs per SM) and every CTA has a tile of the sequence. Measured (bf16, logit
// gates): small training shape, 32 tiles of channels, 8 CTAs 11.5 us against 24.9 us on one;
// long context, 32 tiles, 185 against 675 us; mid-size layer, 256 tiles, 72 us on one CTA
// against 86 us on two.
inline int cluster_ctas(const GatedArgs& a, int tile, int resident) {
    const long long base = (long long)a.B * a.ctiles, most = (long long)resident * sm_count();
    int K = 1;
    while (K < kGatedMaxK && base * 2 * K <= most && (long long)K * tile < a.T) K *= 2;
    return K;
}

template <class Kernel>
lattice_status launch(Kernel k, const GatedArgs& a, int threads, int smem, cudaStream_t st) {
    const long long ctas = (long long)a.B * a.ctiles * a.K;
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.K;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.K > 1 ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k, a);
    return e == cudaSuccess ? LATTICE_OK : cuda_fail(e);
}

template <int I>
using Int = std::integral_constant<int, I>;

// Calls f with the form as a compile-time constant.
template <class F>
lattice_status with_form(int form, F f) {
    switch (form) {
        case 0: return f(Int<0>());
        case 1: return f(Int<1>());
        case 2: return f(Int<2>());
        case 3: return f(Int<3>());
        case 4: return f(Int<4>());
        case 5: return f(Int<5>());
        case 6: return f(Int<6>());
        case 7: return f(Int<7>());
        case 8: return f(Int<8>());
    }
    return LATTICE_ERR_INVALID_ARG;
}

// Calls f with where the gates come from and whether rows are vectors.
template <class XT, class F>
lattice_status with_gates(const GatedArgs& a, bool vec, F f) {
    if (a.zhead) return vec ? f(Int<kZHead>(), std::true_type()) : f(Int<kZHead>(), std::false_type());
    if constexpr (sizeof(XT) == 2) {
        if (a.z32) return vec ? f(Int<kZ32>(), std::true_type()) : f(Int<kZ32>(), std::false_type());
    }
    return vec ? f(Int<kZSame>(), std::true_type()) : f(Int<kZSame>(), std::false_type());
}

// Calls f with a value of x's type.
template <class F>
lattice_status with_type(lattice_dtype t, F f) {
    switch (t) {
        case LATTICE_F32: return f(0.f);
        case LATTICE_BF16: return f(__nv_bfloat16());
        case LATTICE_F16: return f(__half());
    }
    return LATTICE_ERR_INVALID_ARG;
}

}  // namespace gated
}  // namespace lattice

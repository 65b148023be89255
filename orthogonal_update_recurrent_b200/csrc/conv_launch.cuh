// conv_launch.cuh -- launches of the short convolution's kernels (short_conv.cuh), instantiated per
// type of x in conv_*.cu.
#pragma once
#include "launch.h"
#include "short_conv.cuh"

namespace lattice {
namespace conv {

template <class XT, int K, int V>
lattice_status run(const ConvArgs& a, int what, cudaStream_t st) {
    const long long ctas = ((long long)a.B * a.runs * (a.C / V) + 255) / 256;
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    const unsigned n = (unsigned)ctas;
    if (what == kConvFwd) {
        fwd_kernel<XT, K, V><<<n, 256, 0, st>>>(a);
    } else if (what == kConvStep) {
        step_kernel<XT, K, V><<<n, 256, 0, st>>>(a);
    } else {
        bwd_kernel<XT, K, V><<<n, 256, 0, st>>>(a);
        if (a.parts) {
            const lattice_status s = launch_status();
            if (s != LATTICE_OK) return s;
            weights_kernel<<<(unsigned)(((long long)(K + 1) * a.C + 31) / 32), 1024, 0, st>>>(a, (long long)a.B * a.runs);
        }
    }
    return launch_status();
}
template <class XT, int K>
lattice_status run(const ConvArgs& a, int what, int V, cudaStream_t st) {
    return V == 4 ? run<XT, K, 4>(a, what, st) : V == 2 ? run<XT, K, 2>(a, what, st) : run<XT, K, 1>(a, what, st);
}

template <class XT>
lattice_status launch(const ConvArgs& a, int what, int V, cudaStream_t st) {
    switch (a.K) {
        case 1: return run<XT, 1>(a, what, V, st);
        case 2: return run<XT, 2>(a, what, V, st);
        case 3: return run<XT, 3>(a, what, V, st);
        case 4: return run<XT, 4>(a, what, V, st);
        case 5: return run<XT, 5>(a, what, V, st);
        case 6: return run<XT, 6>(a, what, V, st);
        case 7: return run<XT, 7>(a, what, V, st);
        case 8: return run<XT, 8>(a, what, V, st);
    }
    return LATTICE_ERR_UNSUPPORTED;
}

}  // namespace conv
}  // namespace lattice

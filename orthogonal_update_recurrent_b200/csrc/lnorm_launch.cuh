// lnorm_launch.cuh -- launches of the layer norm's kernels (layer_norm.cuh), instantiated per type of
// the call in tu_lnorm_*.cu.
#pragma once
#include "layer_norm.cuh"
#include "norm_launch.cuh"

namespace lattice {
namespace norm {

template <class F, bool SUB, bool BWD>
struct LayerKernel;

template <class F, bool SUB>
lattice_status run_layer(bool bwd, const NormArgs& a, int* groups, cudaStream_t st) {
    // both have the threads of a forward pass
    if (bwd) return launch_kernel<LayerKernel<F, SUB, true>>(layer_bwd_kernel<F, SUB>, false, F::MODE, 96, a, groups, st);
    return launch_kernel<LayerKernel<F, SUB, false>>(layer_fwd_kernel<F, SUB>, false, F::MODE, 64, a, groups, st);
}
template <class T, bool SUB, bool RES, bool Y32, bool R32>
lattice_status run_layer_mode(bool bwd, const NormArgs& a, int mode, int* groups, cudaStream_t st) {
    if (mode == kVec) return run_layer<LayerForm<T, kVec, RES, Y32, R32>, SUB>(bwd, a, groups, st);
    if (mode == kShift) return run_layer<LayerForm<T, kShift, RES, Y32, R32>, SUB>(bwd, a, groups, st);
    return run_layer<LayerForm<T, kOdd, RES, Y32, R32>, SUB>(bwd, a, groups, st);
}
template <class T, bool SUB, bool RES>
lattice_status run_layer_types(bool bwd, const NormArgs& a, int mode, int* groups, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (a.y32) return a.r32 ? run_layer_mode<T, SUB, RES, true, true>(bwd, a, mode, groups, st)
                                : run_layer_mode<T, SUB, RES, true, false>(bwd, a, mode, groups, st);
        return a.r32 ? run_layer_mode<T, SUB, RES, false, true>(bwd, a, mode, groups, st)
                     : run_layer_mode<T, SUB, RES, false, false>(bwd, a, mode, groups, st);
    } else {
        return run_layer_mode<T, SUB, RES, true, true>(bwd, a, mode, groups, st);
    }
}
template <class T>
lattice_status launch_layer(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st) {
    const Split split(a.D, false, mode);
    a.tpr = split.tpr;
    a.K = split.K;
    const bool res = bwd ? a.dr != nullptr : a.residual != nullptr;
    if (a.tpr <= 32) return res ? run_layer_types<T, true, true>(bwd, a, mode, groups, st) : run_layer_types<T, true, false>(bwd, a, mode, groups, st);
    return res ? run_layer_types<T, false, true>(bwd, a, mode, groups, st) : run_layer_types<T, false, false>(bwd, a, mode, groups, st);
}

}  // namespace norm
}  // namespace lattice

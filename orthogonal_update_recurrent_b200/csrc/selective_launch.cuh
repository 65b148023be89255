// selective_launch.cuh -- launches of the selective scan's kernels (selective.cuh, selective_bwd.cuh),
// instantiated per type of x in sel_fwd_*.cu and sel_bwd_*.cu.
#pragma once
#include "launch.h"
#include "selective.cuh"
#include "selective_bwd.cuh"

namespace lattice {
namespace selective {

template <class K>
lattice_status start(K kernel, const SelArgs& a, size_t shared, long long ctas, cudaStream_t st) {
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    if (shared > 48 * 1024) {
        const cudaError_t e = allow_shared(kernel, shared);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    kernel<<<(unsigned)ctas, NT, shared, st>>>(a);
    return launch_status();
}
inline long long ctas_of(const SelArgs& a) { return (long long)a.B * a.nseg * a.G * a.tiles; }

template <class XT, int L, int S, bool VEC>
lattice_status forward_(const SelArgs& a, cudaStream_t st) {
    if (a.nseg > 1) {
        lattice_status s = start(seg_kernel<XT, L, S, false, VEC>, a, sizeof(SegShared<XT, L, S>), ctas_of(a), st);
        if (s != LATTICE_OK) return s;
        s = start(join_kernel<false>, a, 0, ((long long)a.B * a.E * a.N + 255) / 256, st);
        if (s != LATTICE_OK) return s;
    }
    return start(fwd_kernel<XT, L, S, VEC>, a, sizeof(FwdShared<XT, L, S>), ctas_of(a), st);
}

template <class XT, int L, int S>
lattice_status forward(const SelArgs& a, cudaStream_t st) {
    return a.vec ? forward_<XT, L, S, true>(a, st) : forward_<XT, L, S, false>(a, st);
}

template <class XT, int L, bool VEC>
lattice_status backward_(const SelArgs& a, cudaStream_t st) {
    lattice_status s = LATTICE_OK;
    if (a.nseg > 1) {
        s = start(seg_kernel<XT, L, 4, true, VEC>, a, sizeof(SegShared<XT, L, 4>), ctas_of(a), st);
        if (s != LATTICE_OK) return s;
        s = start(join_kernel<true>, a, 0, ((long long)a.B * a.E * a.N + 255) / 256, st);
        if (s != LATTICE_OK) return s;
    }
    s = a.z ? start(bwd_kernel<XT, L, true, VEC>, a, sizeof(BwdShared<XT, L>), ctas_of(a), st)
            : start(bwd_kernel<XT, L, false, VEC>, a, sizeof(BwdShared<XT, L>), ctas_of(a), st);
    if (s != LATTICE_OK) return s;
    if (a.T > 0) {
        s = start(shared_kernel<XT>, a, 0, ((long long)a.B * a.T * a.G * 2 * a.N + 255) / 256, st);
        if (s != LATTICE_OK) return s;
    }
    return start(weights_kernel, a, 0, ((long long)a.E * a.N + 2 * a.E + 255) / 256, st);
}

template <class XT, int L>
lattice_status backward(const SelArgs& a, cudaStream_t st) {
    return a.vec ? backward_<XT, L, true>(a, st) : backward_<XT, L, false>(a, st);
}

// Four sequences per thread where enough threads are left to fill the device with 16 warps per SM
template <class XT, int L>
lattice_status one_token(const SelArgs& a, cudaStream_t st) {
    auto ctas = [&](int R) { return (a.B + (long long)R - 1) / R * (((long long)a.E * L + 255) / 256); };
    const bool many = ctas(4) >= 2 * sm_count();
    if (a.vec) return many ? start(step_kernel<XT, L, 4, true>, a, 0, ctas(4), st) : start(step_kernel<XT, L, 1, true>, a, 0, ctas(1), st);
    return many ? start(step_kernel<XT, L, 4, false>, a, 0, ctas(4), st) : start(step_kernel<XT, L, 1, false>, a, 0, ctas(1), st);
}

template <class XT>
lattice_status launch_fwd(const SelArgs& a, int S, cudaStream_t st) {
    switch (sel_padded(a.N)) {
        case 8: return S == 2 ? forward<XT, 4, 2>(a, st) : forward<XT, 2, 4>(a, st);
        case 16: return S == 2 ? forward<XT, 8, 2>(a, st) : forward<XT, 4, 4>(a, st);
        case 32: return S == 2 ? forward<XT, 16, 2>(a, st) : forward<XT, 8, 4>(a, st);
        case 64: return forward<XT, 16, 4>(a, st);
        default: return forward<XT, 32, 4>(a, st);
    }
}
template <class XT>
lattice_status launch_bwd(const SelArgs& a, cudaStream_t st) {
    switch (sel_padded(a.N)) {
        case 8: return backward<XT, 2>(a, st);
        case 16: return backward<XT, 4>(a, st);
        case 32: return backward<XT, 8>(a, st);
        case 64: return backward<XT, 16>(a, st);
        default: return backward<XT, 32>(a, st);
    }
}
template <class XT>
lattice_status launch_step(const SelArgs& a, cudaStream_t st) {
    if (a.N <= 4) return one_token<XT, 1>(a, st);
    switch (sel_padded(a.N)) {
        case 8: return one_token<XT, 2>(a, st);
        case 16: return one_token<XT, 4>(a, st);
        case 32: return one_token<XT, 8>(a, st);
        case 64: return one_token<XT, 16>(a, st);
        default: return one_token<XT, 32>(a, st);
    }
}

}  // namespace selective
}  // namespace lattice

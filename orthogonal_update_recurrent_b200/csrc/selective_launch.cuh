// selective_launch.cuh -- launches of the selective scan's kernels (selective.cuh, selective_bwd.cuh),
// instantiated per type of x in sel_fwd_*.cu and sel_bwd_*.cu.
#pragma once
#include "launch.h"
#include "selective.cuh"
#include "selective_bwd.cuh"

namespace lattice {
namespace selective {

template <class K>
lattice_status start(K kernel, const SelArgs& a, int threads, size_t shared, long long ctas, cudaStream_t st) {
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    if (shared > 48 * 1024) {
        const cudaError_t e = allow_shared(kernel, shared);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    kernel<<<(unsigned)ctas, (unsigned)threads, shared, st>>>(a);
    return launch_status();
}
inline long long ctas_of(const SelArgs& a) { return (long long)a.B * a.nseg * a.G * a.tiles; }

template <class XT, int L, int S, int W, bool VEC>
lattice_status forward(const SelArgs& a, cudaStream_t st) {
    if (a.nseg > 1) {
        lattice_status s = start(seg_kernel<XT, L, S, W, false, VEC>, a, 32 * W, sizeof(SegShared<XT, L, S, W>), ctas_of(a), st);
        if (s != LATTICE_OK) return s;
        if (a.joined) s = start(join_kernel<false>, a, 256, 0, ((long long)a.B * a.E * a.N + 255) / 256, st);
        if (s != LATTICE_OK) return s;
    }
    return start(fwd_kernel<XT, L, S, W, VEC>, a, 32 * W, sizeof(FwdShared<XT, L, S, W>), ctas_of(a), st);
}
template <class XT, int L, int S>
lattice_status forward(const SelArgs& a, int W, cudaStream_t st) {
    if (W == 2) return a.vec ? forward<XT, L, S, 2, true>(a, st) : forward<XT, L, S, 2, false>(a, st);
    return a.vec ? forward<XT, L, S, 8, true>(a, st) : forward<XT, L, S, 8, false>(a, st);
}

template <class XT, int L, int W, bool VEC>
lattice_status backward(const SelArgs& a, cudaStream_t st) {
    lattice_status s = LATTICE_OK;
    if (a.nseg > 1) {
        s = start(seg_kernel<XT, L, 4, W, true, VEC>, a, 32 * W, sizeof(SegShared<XT, L, 4, W>), ctas_of(a), st);
        if (s != LATTICE_OK) return s;
        if (a.joined) s = start(join_kernel<true>, a, 256, 0, ((long long)a.B * a.E * a.N + 255) / 256, st);
        if (s != LATTICE_OK) return s;
    }
    s = a.z ? start(bwd_kernel<XT, L, W, true, VEC>, a, 32 * W, sizeof(BwdShared<XT, L, W>), ctas_of(a), st)
            : start(bwd_kernel<XT, L, W, false, VEC>, a, 32 * W, sizeof(BwdShared<XT, L, W>), ctas_of(a), st);
    if (s != LATTICE_OK) return s;
    int width = 2;
    while (width < 2 * a.N) width *= 2;
    long long tokens = (long long)a.B * a.T / (16 * sm_count());  // several CTAs per SM, none with more than 64 tokens
    const int least = 256 / width / a.G;
    tokens = tokens > 64 ? 64 : tokens < least ? least : tokens < 1 ? 1 : tokens;
    const long long most = a.T > 0 ? a.B * ((a.T + tokens - 1) / tokens) : 0, ctas = most + (sel_columns(a.E, a.N) + 31) / 32;
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    sums_kernel<XT><<<(unsigned)ctas, 256, 0, st>>>(a, width, (int)tokens, (int)most);
    return launch_status();
}
template <class XT, int L>
lattice_status backward(const SelArgs& a, int W, cudaStream_t st) {
    if (W == 2) return a.vec ? backward<XT, L, 2, true>(a, st) : backward<XT, L, 2, false>(a, st);
    return a.vec ? backward<XT, L, 8, true>(a, st) : backward<XT, L, 8, false>(a, st);
}

// Four sequences per thread where enough threads are left to fill the device with 16 warps per SM
template <class XT, int L>
lattice_status one_token(const SelArgs& a, cudaStream_t st) {
    auto ctas = [&](int R) { return (a.B + (long long)R - 1) / R * (((long long)a.E * L + 255) / 256); };
    const bool many = ctas(4) >= 2 * sm_count();
    if (a.vec) return many ? start(step_kernel<XT, L, 4, true>, a, 256, 0, ctas(4), st) : start(step_kernel<XT, L, 1, true>, a, 256, 0, ctas(1), st);
    return many ? start(step_kernel<XT, L, 4, false>, a, 256, 0, ctas(4), st) : start(step_kernel<XT, L, 1, false>, a, 256, 0, ctas(1), st);
}

template <class XT>
lattice_status launch_fwd(const SelArgs& a, int S, int W, cudaStream_t st) {
    switch (sel_padded(a.N)) {
        case 8: return S == 2 ? forward<XT, 4, 2>(a, W, st) : forward<XT, 2, 4>(a, W, st);
        case 16: return S == 2 ? forward<XT, 8, 2>(a, W, st) : forward<XT, 4, 4>(a, W, st);
        case 32: return S == 2 ? forward<XT, 16, 2>(a, W, st) : forward<XT, 8, 4>(a, W, st);
        case 64: return forward<XT, 16, 4>(a, W, st);
        default: return forward<XT, 32, 4>(a, W, st);
    }
}
template <class XT>
lattice_status launch_bwd(const SelArgs& a, int W, cudaStream_t st) {
    switch (sel_padded(a.N)) {
        case 8: return backward<XT, 2>(a, W, st);
        case 16: return backward<XT, 4>(a, W, st);
        case 32: return backward<XT, 8>(a, W, st);
        case 64: return backward<XT, 16>(a, W, st);
        default: return backward<XT, 32>(a, W, st);
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

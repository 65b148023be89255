// gated_fwd_launch.cuh -- launches of the gated recurrence's forward and single-token kernels
// (gated.cuh), instantiated per type of x in tu_gated_fwd_*.cu.
#pragma once
#include "gated_launch.cuh"

namespace lattice {
namespace gated {

// Two channels per lane; runs of 16 tokens on 8 warps, two CTAs per SM (mid-size layer, bf16:
// 78 us, 74 us since; runs of 8 on three CTAs 86 us: a run's exchange is then spread over half the
// elements). fp32 rows are twice as wide, so runs of 8 keep the stages as large.
template <class XT, int FORM, int ZM, int ROWS>
lattice_status fwd(GatedArgs a, cudaStream_t st) {
    constexpr int V = kGatedFwdVec, NW = 8, R = sizeof(XT) == 2 ? 16 : 8, NST = ZM == kZHead ? 3 : 2, MINB = R == 16 ? 2 : 3;
    static_assert(FwdLayout<XT, ZM, ROWS, V, R, NW, NST>::bytes(8) <= kMaxShared, "clusters of 8 fit");
    a.ctiles = (a.C + 32 * V - 1) / (32 * V);
    return launch(gated_fwd_kernel<XT, ZM, FORM, ROWS, V, R, NW, NST, MINB>, a, NW * 32, NW * R, MINB,
                  [](int K) { return FwdLayout<XT, ZM, ROWS, V, R, NW, NST>::bytes(K); }, st);
}

template <class XT, int FORM, int ZM, bool VEC>
lattice_status step(const GatedArgs& a, cudaStream_t st) {
    const long long threads = (long long)a.B * ((a.C + kStepVec - 1) / kStepVec), ctas = (threads + 255) / 256;
    if (ctas > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    gated_step_kernel<XT, ZM, FORM, VEC, kStepVec><<<(unsigned)ctas, 256, 0, st>>>(a);
    return launch_status();
}

template <class XT>
lattice_status launch_fwd(GatedArgs a, int form, bool vec, cudaStream_t st) {
    return with_form(form, [&](auto f) {
        return with_gates<XT>(a, vec ? a.wide ? kWide : kPairs : kAny, [&](auto zm, auto v) {
            return fwd<XT, decltype(f)::value, decltype(zm)::value, decltype(v)::value>(a, st);
        });
    });
}

template <class XT>
lattice_status launch_step(const GatedArgs& a, int form, bool vec, cudaStream_t st) {
    return with_form(form, [&](auto f) {
        return with_gates<XT>(a, vec ? kPairs : kAny, [&](auto zm, auto v) {
            return step<XT, decltype(f)::value, decltype(zm)::value, decltype(v)::value != kAny>(a, st);
        });
    });
}

}  // namespace gated
}  // namespace lattice

// gated_bwd_launch.cuh -- launches of the gated recurrence's backward kernel (gated.cuh),
// instantiated per type of x in tu_gated_bwd_*.cu.
#pragma once
#include "gated_launch.cuh"

namespace lattice {
namespace gated {

template <class XT, int FORM, int ZM, int ROWS, int V, int NW, int NST, int MINB>
lattice_status bwd_of(GatedArgs a, cudaStream_t st) {
    constexpr int R = kGatedMark;
    static_assert(BwdLayout<XT, ZM, ROWS, V, R, NW, NST>::bytes(8) <= kMaxShared, "clusters of 8 fit");
    a.ctiles = (a.C + 32 * V - 1) / (32 * V);
    return launch(gated_bwd_kernel<XT, ZM, FORM, ROWS, V, R, NW, NST, MINB>, a, NW * 32, NW * R, MINB,
                  [](int K) { return BwdLayout<XT, ZM, ROWS, V, R, NW, NST>::bytes(K); }, st);
}

// Gates per channel: two channels per lane, 4 warps, two CTAs per SM. Gates per head: four
// channels per lane, so that a warp's 128 channels hold whole heads (d <= 128) and a head's
// gradient is summed within it; 8 warps (mid-size layer 90 us, 4 warps 106 us), 4 for fp32,
// whose stages are twice as large. fp32 heads of up to 64 have two channels per lane, as gates
// per channel (5 x 3 heads of 64, 1531 tokens: 14.5 us against 16.5 us; in 16 bits slower, 4 x 28 heads
// of 64, 4681 tokens: 86 us against 70 us).
template <class XT, int FORM, int ZM, int ROWS>
lattice_status bwd(const GatedArgs& a, cudaStream_t st) {
    if constexpr (ZM == kZHead && sizeof(XT) == 4)
        if (a.d <= 32 * kGatedBwdVec) return bwd_of<XT, FORM, ZM, ROWS, kGatedBwdVec, 4, 2, 2>(a, st);
    if constexpr (ZM == kZHead) return bwd_of<XT, FORM, ZM, ROWS, kGatedHeadVec, sizeof(XT) == 2 ? 8 : 4, 2, 1>(a, st);
    else return bwd_of<XT, FORM, ZM, ROWS, kGatedBwdVec, 4, 2, 2>(a, st);
}

template <class XT>
lattice_status launch_bwd(GatedArgs a, int form, bool vec, cudaStream_t st) {
    return with_form(form, [&](auto f) {
        return with_gates<XT>(a, vec ? a.wide ? kWide : kPairs : kAny, [&](auto zm, auto v) {
            return bwd<XT, decltype(f)::value, decltype(zm)::value, decltype(v)::value>(a, st);
        });
    });
}

}  // namespace gated
}  // namespace lattice

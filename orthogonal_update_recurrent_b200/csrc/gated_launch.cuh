// gated_launch.cuh -- what the launches of the gated recurrence's two directions share.
#pragma once
#include <atomic>
#include <type_traits>

#include "gated.cuh"
#include "launch.h"

namespace lattice {
namespace gated {

// Launches `base` clusters of K CTAs, a.B * a.ctiles of them: the largest K with which all are
// resident at once (up to `resident` CTAs per SM) and every CTA has a tile of the sequence.
// Clusters lie within a GPC, which may hold fewer of a size than its SMs would, so the device
// is asked (once per kernel, size and device). Measured (bf16, logit gates): small training
// shape, 32 tiles of channels, 8 CTAs 11.8 us against 26.9 us on one; 50 tiles of 8192
// tokens, 5 CTAs 43 us, 4 50 us, 6 (not all resident) 58 us; mid-size layer, 256 tiles,
// 78 us on one CTA against 86 us on two (74 us since). More than 8 CTAs, where the device allows them, serve few
// channels over long sequences: 256 channels of 20000 tokens, tau 1/16 and unit write, 16 CTAs
// 49 us, 8 86 us (16 41 us since).
constexpr int kMaxDevices = 16;
constexpr int kMaxShared = 227 * 1024;  // bytes of shared memory a CTA may have

template <class Kernel, class Bytes>
lattice_status launch(Kernel k, GatedArgs a, int threads, int tile, int resident, Bytes bytes, cudaStream_t st) {
    static std::atomic<int> held[kMaxDevices][kGatedMaxK + 1];  // clusters of a size that the device holds, plus 1
    const long long base = (long long)a.B * a.ctiles;
    long long K = (long long)resident * sm_count() / base;
    if (K > kGatedMaxK) K = kGatedMaxK;
    if (K > ((long long)a.T + tile - 1) / tile) K = ((long long)a.T + tile - 1) / tile;
    if (K < 1) K = 1;
    int most = kGatedMaxK;  // the largest K whose shared memory a CTA may have
    while (bytes(most) > kMaxShared) --most;
    if (K > most) K = most;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    for (;; --K) {
        a.K = (int)K;
        const int smem = bytes(a.K);
        if (smem > 40 * 1024) {
            e = allow_shared(k, bytes(most));
            if (e != cudaSuccess) return cuda_fail(e);
        }
        if (K > 8) {  // above the portable size
            e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return cuda_fail(e);
        }
        cfg.dynamicSmemBytes = smem;
        attr[0].val.clusterDim.x = (unsigned)K;
        cfg.numAttrs = K > 1 ? 1 : 0;
        if (base * K > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
        cfg.gridDim = dim3((unsigned)(base * K));
        if (K == 1) break;
        int n = dev < kMaxDevices ? held[dev][K].load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
            if (e != cudaSuccess) return cuda_fail(e);
            ++n;
            if (dev < kMaxDevices) held[dev][K].store(n, std::memory_order_relaxed);
        }
        if (n - 1 >= base) break;
    }
    e = cudaLaunchKernelEx(&cfg, k, a);
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

// Calls f with where the gates come from and how rows start.
template <class XT, class F>
lattice_status with_gates(const GatedArgs& a, int rows, F f) {
    auto g = [&](auto zm) {
        return rows == kWide ? f(zm, Int<kWide>()) : rows == kPairs ? f(zm, Int<kPairs>()) : f(zm, Int<kAny>());
    };
    if (a.zhead) return g(Int<kZHead>());
    if constexpr (sizeof(XT) == 2) {
        if (a.z32) return g(Int<kZ32>());
    }
    return g(Int<kZSame>());
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

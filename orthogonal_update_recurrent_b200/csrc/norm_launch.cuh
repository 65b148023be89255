// norm_launch.cuh -- launches of the block norms' kernels (block_norm.cuh), instantiated per
// type of the call in tu_norm_*.cu.
#pragma once
#include <atomic>

#include "block_norm.cuh"
#include "launch.h"

namespace lattice {
namespace norm {

inline int most_threads(bool bwd, int mode) { return bwd ? kBwdThreads : mode != kOdd ? kFwdThreads : kFwdOddThreads; }
// Rows after which they start at the same place among 8 elements again.
inline int period(int D) { return D % 8 == 0 ? 1 : D % 4 == 0 ? 2 : D % 2 == 0 ? 4 : 8; }

// 8 elements per thread: a row's CTAs (1, 2 or 4) and its threads in each, a power of two
// within a warp and whole warps above. Shifted vectors (kShift) start up to `shift` early.
struct Split {
    int K, tpr, threads, rows;  // threads of a CTA, rows that it takes at once
    int most, resident;
    Split(int D, bool bwd, int mode) : K(1), most(most_threads(bwd, mode)), resident(bwd ? kBwdThreads : kFwdThreads) {
        const int shift = mode == kShift ? 8 - 8 / period(D) : 0;
        while (K * most * 8 < D + shift) K *= 2;
        const int need = (D + shift + 8 * K - 1) / (8 * K);
        tpr = 1;
        if (need > 32) tpr = (need + 31) / 32 * 32;
        else
            while (tpr < need) tpr *= 2;
        threads = tpr > 32 ? tpr : 256;
        rows = threads / tpr;
    }
    // groups of K CTAs that take N rows: at most what `resident` threads per SM are
    long long groups(long long N) const {
        const long long turns = (N + rows - 1) / rows, at_once = (long long)sm_count() * (resident / threads) / K;
        return turns < at_once ? turns : at_once;
    }
    // n of them, rounded so that those with several turns step by whole periods
    long long whole_periods(long long n, long long N, int D) const {
        const long long turns = (N + rows - 1) / rows, p = period(D);
        if (n >= turns || rows % p == 0) return n;
        return n >= p ? n / p * p : p < turns ? p : turns;
    }
};

// The grid is what the device holds at once, or fewer: it is asked once per kernel, CTA size and
// device. (Clusters lie within a GPC, which may hold fewer than its SMs would: 4096 rows of
// 16384, backward: 543 us with a cluster of 4 for every 4 SMs, 316 us with as many as are held.)
constexpr int kMaxDevices = 16;

template <class F, bool SUB, bool BWD>  // names the kernel: all of them have one type
lattice_status launch(const NormArgs& a, int* groups, cudaStream_t st) {
    constexpr int mode = F::MODE, bytes_per_thread = BWD ? 128 : 64;
    void (*k)(NormArgs);
    if constexpr (BWD) k = norm_bwd_kernel<F, SUB>;
    else k = norm_fwd_kernel<F, SUB>;
    const Split split(a.D, BWD, mode);
    const int threads = split.threads, smem = threads * bytes_per_thread;
    cudaError_t e;
    if (smem > 40 * 1024) {  // 48 KB with the static arrays
        e = allow_shared(k, (size_t)split.most * bytes_per_thread);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.K);
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
    static std::atomic<int> held[kMaxDevices][33][3];  // of this kernel, by warps of a CTA, and K: 1, 2, 4
    int dev = 0, c = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    std::atomic<int>* slot = dev < kMaxDevices ? &held[dev][threads / 32][a.K / 2] : nullptr;
    if (slot) c = slot->load(std::memory_order_relaxed);
    if (c == 0) {
        e = a.K > 1 ? cudaOccupancyMaxActiveClusters(&c, k, &cfg)
                    : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&c, k, threads, smem);
        if (e != cudaSuccess) return cuda_fail(e);
        if (a.K == 1) c *= sm_count();
        if (c < 1) return LATTICE_ERR_UNSUPPORTED;
        if (slot) slot->store(c, std::memory_order_relaxed);
    }
    long long n = split.groups(a.N);
    if (n > c) n = c;
    if (mode == kShift) n = split.whole_periods(n, a.N, a.D);
    cfg.gridDim = dim3((unsigned)(n * a.K));
    if (groups) *groups = (int)n;
    e = cudaLaunchKernelEx(&cfg, k, a);
    return e == cudaSuccess ? LATTICE_OK : cuda_fail(e);
}

template <class F, bool SUB>
lattice_status run(bool bwd, const NormArgs& a, int* groups, cudaStream_t st) {
    return bwd ? launch<F, SUB, true>(a, groups, st) : launch<F, SUB, false>(a, groups, st);
}

template <class T, bool SUB, bool GATE, int Y32, int R32>
lattice_status run_typed(bool bwd, const NormArgs& a, int mode, int* groups, cudaStream_t st) {
    const bool pre = bwd ? a.dn != nullptr : a.n_out != nullptr;
    if (mode == kOdd) return run<Form<T, kOdd, GATE, Y32, R32, -1>, SUB>(bwd, a, groups, st);
    if (mode == kShift)
        return pre ? run<Form<T, kShift, GATE, Y32, R32, 1>, SUB>(bwd, a, groups, st)
                   : run<Form<T, kShift, GATE, Y32, R32, 0>, SUB>(bwd, a, groups, st);
    return pre ? run<Form<T, kVec, GATE, Y32, R32, 1>, SUB>(bwd, a, groups, st)
               : run<Form<T, kVec, GATE, Y32, R32, 0>, SUB>(bwd, a, groups, st);
}

template <class T, bool SUB, bool GATE>
lattice_status run_types(bool bwd, const NormArgs& a, int mode, int* groups, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (a.y32)
            return a.r32 ? run_typed<T, SUB, GATE, 1, 1>(bwd, a, mode, groups, st) : run_typed<T, SUB, GATE, 1, 0>(bwd, a, mode, groups, st);
        return a.r32 ? run_typed<T, SUB, GATE, 0, 1>(bwd, a, mode, groups, st) : run_typed<T, SUB, GATE, 0, 0>(bwd, a, mode, groups, st);
    } else {
        return run_typed<T, SUB, GATE, 1, 1>(bwd, a, mode, groups, st);
    }
}

template <class T>
lattice_status launch_norm(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st) {
    const Split split(a.D, bwd, mode);
    a.tpr = split.tpr;
    a.K = split.K;
    if (a.tpr <= 32) return a.gate ? run_types<T, true, true>(bwd, a, mode, groups, st) : run_types<T, true, false>(bwd, a, mode, groups, st);
    return a.gate ? run_types<T, false, true>(bwd, a, mode, groups, st) : run_types<T, false, false>(bwd, a, mode, groups, st);
}

}  // namespace norm
}  // namespace lattice

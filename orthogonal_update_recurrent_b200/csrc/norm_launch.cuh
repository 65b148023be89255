// norm_launch.cuh -- launches of the block norms' kernels (block_norm.cuh), instantiated per
// type of the call in tu_norm_*.cu.
#pragma once
#include "block_norm.cuh"
#include "launch.h"

namespace lattice {
namespace norm {

// 64 and 128 registers per thread: threads of a CTA at most, and resident on an SM.
constexpr int kFwdThreads = 1024, kBwdThreads = 512;
inline int most_threads(bool bwd) { return bwd ? kBwdThreads : kFwdThreads; }

// 8 elements per thread: a row's CTAs (1, 2 or 4) and its threads in each, a power of two
// within a warp and whole warps above.
struct Split {
    int K, tpr, threads, rows;  // threads of a CTA, rows that it takes at once
    Split(int D, bool bwd) : K(1) {
        while (K * most_threads(bwd) * 8 < D) K *= 2;
        const int need = (D + 8 * K - 1) / (8 * K);
        tpr = 1;
        if (need > 32) tpr = (need + 31) / 32 * 32;
        else
            while (tpr < need) tpr *= 2;
        threads = tpr > 32 ? tpr : 256;
        rows = threads / tpr;
    }
    // groups of K CTAs that take N rows: as many as are resident at once, or fewer
    long long groups(long long N, bool bwd) const {
        const long long turns = (N + rows - 1) / rows, most = (long long)sm_count() * (most_threads(bwd) / threads) / K;
        return turns < most ? turns : most;
    }
};

template <class Kernel>
lattice_status launch(Kernel k, const NormArgs& a, bool bwd, int bytes_per_thread, cudaStream_t st) {
    const Split split(a.D, bwd);
    const int threads = split.threads, smem = threads * bytes_per_thread;
    if (smem > 40 * 1024) {  // 48 KB with the static arrays
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split.groups(a.N, bwd) * split.K));
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

template <class F, bool SUB>
lattice_status run(bool bwd, const NormArgs& a, cudaStream_t st) {
    return bwd ? launch(norm_bwd_kernel<F, SUB>, a, true, 128, st) : launch(norm_fwd_kernel<F, SUB>, a, false, 64, st);
}

template <class T, bool SUB, bool GATE, int Y32, int R32>
lattice_status run_vec(bool bwd, const NormArgs& a, cudaStream_t st) {
    return (bwd ? a.dn : a.n_out) ? run<Form<T, 8, GATE, Y32, R32, 1>, SUB>(bwd, a, st)
                                  : run<Form<T, 8, GATE, Y32, R32, 0>, SUB>(bwd, a, st);
}

template <class T, bool SUB, bool GATE>
lattice_status run_types(bool bwd, const NormArgs& a, bool vec, cudaStream_t st) {
    if (!vec) return run<Form<T, 1, GATE, -1, -1, -1>, SUB>(bwd, a, st);
    if constexpr (sizeof(T) == 2) {
        if (a.y32) return a.r32 ? run_vec<T, SUB, GATE, 1, 1>(bwd, a, st) : run_vec<T, SUB, GATE, 1, 0>(bwd, a, st);
        return a.r32 ? run_vec<T, SUB, GATE, 0, 1>(bwd, a, st) : run_vec<T, SUB, GATE, 0, 0>(bwd, a, st);
    } else {
        return run_vec<T, SUB, GATE, 1, 1>(bwd, a, st);
    }
}

template <class T>
lattice_status launch_norm(bool bwd, NormArgs a, bool vec, cudaStream_t st) {
    const Split split(a.D, bwd);
    a.tpr = split.tpr;
    a.K = split.K;
    if (a.tpr <= 32) return a.gate ? run_types<T, true, true>(bwd, a, vec, st) : run_types<T, true, false>(bwd, a, vec, st);
    return a.gate ? run_types<T, false, true>(bwd, a, vec, st) : run_types<T, false, false>(bwd, a, vec, st);
}

}  // namespace norm
}  // namespace lattice

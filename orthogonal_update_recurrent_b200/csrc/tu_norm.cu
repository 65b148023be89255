// tu_norm.cu -- launches of the block norms' kernels (block_norm.cuh).
#include "block_norm.cuh"
#include "common.cuh"
#include "launch.h"

namespace lattice {
namespace {

// Threads per row for `per` elements each, a power of two.
int threads_per_row(int D, int per) {
    int t = 1;
    while (t * per < D) t *= 2;
    return t;
}
// Elements per thread. Forward: 8, 16 above 8192. Backward, which holds about ten values per
// element: 8 up to 2048, 16 up to 8192, then 32.
int fwd_per(int D) { return D <= 8192 ? 8 : 16; }
int bwd_per(int D) { return D <= 2048 ? 8 : D <= 8192 ? 16 : 32; }

template <class XT, bool CTA, int V, int NV>
lattice_status fwd(const NormArgs& a, cudaStream_t st) {
    const int threads = CTA ? a.tpr : 256, rows = threads / a.tpr;
    const long long turns = (a.N + rows - 1) / rows, most = (long long)sm_count() * (2048 / threads);
    norm::norm_fwd_kernel<XT, CTA, V, NV><<<(unsigned)(turns < most ? turns : most), threads, 0, st>>>(a);
    return launch_status();
}

template <class XT, bool CTA, int V, int NV>
lattice_status bwd(const NormArgs& a, cudaStream_t st) {
    const int threads = CTA ? a.tpr : 256;
    norm::norm_bwd_kernel<XT, CTA, V, NV><<<(unsigned)norm_parts(a.N, a.D), threads, 0, st>>>(a);
    return launch_status();
}

template <class F>
lattice_status with_type(lattice_dtype t, F f) {
    return t == LATTICE_F32 ? f(0.f) : t == LATTICE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

}  // namespace

// CTAs of the backward kernel: as many as are resident at once, or fewer.
int norm_parts(long long N, int D) {
    const int tpr = threads_per_row(D, bwd_per(D)), threads = tpr > 32 ? tpr : 256, rows = threads / tpr;
    const long long turns = (N + rows - 1) / rows, most = (long long)sm_count() * (512 / threads);
    return (int)(turns < most ? turns : most);
}

lattice_status launch_norm_fwd(NormArgs a, lattice_dtype dtype, bool vec, cudaStream_t st) {
    a.tpr = threads_per_row(a.D, fwd_per(a.D));
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (fwd_per(a.D) == 16) return vec ? fwd<T, true, 8, 2>(a, st) : fwd<T, true, 1, 16>(a, st);
        if (a.tpr > 32) return vec ? fwd<T, true, 8, 1>(a, st) : fwd<T, true, 1, 8>(a, st);
        return vec ? fwd<T, false, 8, 1>(a, st) : fwd<T, false, 1, 8>(a, st);
    });
}

lattice_status launch_norm_bwd(NormArgs a, lattice_dtype dtype, bool vec, float* dw_post, float* dw_pre, cudaStream_t st) {
    const int per = bwd_per(a.D);
    a.tpr = threads_per_row(a.D, per);
    const lattice_status s = with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (per == 32) return vec ? bwd<T, true, 8, 4>(a, st) : bwd<T, true, 1, 32>(a, st);
        if (per == 16) return vec ? bwd<T, true, 8, 2>(a, st) : bwd<T, true, 1, 16>(a, st);
        if (a.tpr > 32) return vec ? bwd<T, true, 8, 1>(a, st) : bwd<T, true, 1, 8>(a, st);
        return vec ? bwd<T, false, 8, 1>(a, st) : bwd<T, false, 1, 8>(a, st);
    });
    if (s != LATTICE_OK || !a.parts) return s;
    norm::norm_dw_kernel<<<(unsigned)((2 * a.D + 31) / 32), 256, 0, st>>>(a.parts, norm_parts(a.N, a.D), a.D, a.scale, dw_post,
                                                                        dw_pre);
    return launch_status();
}

cudaError_t status_norm(unsigned int* v) { return read_clear_module_status(v); }

}  // namespace lattice

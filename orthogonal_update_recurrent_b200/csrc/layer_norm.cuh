// layer_norm.cuh -- layer norm of rows, with the residual that they are added to first, and its
// backward pass (sm_100a).
//
// Per row of D elements:
//   r = residual + x (rounded to the residual's type, or r = x), u = r - mean r, rho = 1/sqrt(mean u^2 + eps)
//   n = u rho w + b
// Backward, from dn and dr, with m = w dn:
//   d r = dr + rho (m - mean m - u rho^2 mean(m u)),  dw = sum over rows of dn u rho,  db = sum over rows of dn
//
// HBM bounds both. Rows are read, summed and kept in registers as in the norms after and before a
// block (block_norm.cuh, whose threads, columns and row sums these kernels use). The mean is taken
// first and the variance from the differences: a large mean costs no more than the roundings of its own sum. The
// second sum costs an exchange more, during which the next row is on its way. What is left is bound by
// those exchanges, so both directions keep 1024 threads' rows at once per SM, 64 registers each. (One exchange of
// differences from the row's first element, a second one where that cancels, was slower: 32768 rows of 2048 bf16, no residual,
// forward 62 -> 84 us.) 32768 rows of 2048, bf16 with residual and r in fp32: 131 us forward, 6.1 TB/s; backward 185 us, 5.8 TB/s, and 4 us for
// the weights' sums.
#pragma once
#include "block_norm.cuh"

namespace lattice {
namespace norm {

// The thread's columns that are the row's own, a bit each.
template <int MODE>
__device__ __forceinline__ unsigned own_columns(const Columns<MODE>& c) {
    unsigned m = 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        const int at = MODE == kOdd ? c.at(v) : c.first + v;
        m |= ((unsigned)at < (unsigned)c.D ? 1u : 0u) << v;
    }
    return m;
}
// sum / D to within one rounding: 1/D in two parts (inv_d + inv_d_rest, off by 2^-48 of it) times the sum, whose product's own rounding is
// added back. A rounded 1/D alone leaves a constant row of 1000 a deviation of 6e-5, which 1/sqrt(eps) raises to 0.02. (A division,
// whose general case is a call, spills the rows' registers: 32768 rows of 2048 bf16, fp32 residual, backward 186 -> 215 us.)
__device__ __forceinline__ float mean_of(const NormArgs& A, float sum) {
    const float m = __fmul_rn(sum, A.inv_d);
    return __fadd_rn(m, fmaf(sum, A.inv_d_rest, fmaf(sum, A.inv_d, -m)));
}
// u = r - mean, 0 in columns of other rows
__device__ __forceinline__ void centre(const F2* r, float mean, unsigned mine, F2* u) {
#pragma unroll
    for (int v = 0; v < 4; ++v) u[v] = add2(r[v], f2(-mean));
    if (mine == 0xffu) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        float a, b;
        parts(u[v], a, b);
        u[v] = f2(mine & (1u << (2 * v)) ? a : 0.f, mine & (2u << (2 * v)) ? b : 0.f);
    }
}
__device__ __forceinline__ float sum8(const F2* a) { return both(add2(add2(a[0], a[1]), add2(a[2], a[3]))); }

// The columns' weights into the thread's shared memory: `none` where w is null, 0 in columns of other rows
template <class XT, int MODE>
__device__ __forceinline__ void keep_columns(const void* w, bool w32, float none, const Columns<MODE>& c, unsigned mine, ulonglong2* to) {
    float t[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        t[v] = 0.f;
        if (!(mine & (1u << v))) continue;
        t[v] = none;
        if (w) values<XT, 1>(load<XT, 1>(w, w32, MODE == kOdd ? c.at(v) : c.first + v), w32, t + v);
    }
    const F2 f[4] = {f2(t[0], t[1]), f2(t[2], t[3]), f2(t[4], t[5]), f2(t[6], t[7])};
    own_write(to, f);
}
// The values as they are after rounding to XT
template <class XT>
__device__ __forceinline__ void rounded(F2* f) {
    if constexpr (sizeof(XT) == 2) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float a, b;
            parts(f[v], a, b);
            unpack(XT(), pack(XT(), a, b), a, b);
            f[v] = f2(a, b);
        }
    }
}

// RES: with a residual. Y32, R32: x; residual and r (backward: r and dr) are fp32. In A: y is x
// (backward: r), w_post and w_pre are w and b.
template <class XT_, int MODE_, bool RES_, bool Y32_, bool R32_>
struct LayerForm {
    using XT = XT_;
    static constexpr int MODE = MODE_, V = MODE == kOdd ? 1 : 8;
    static constexpr bool RES = RES_, Y32 = Y32_, R32 = R32_;
};

template <class F, bool SUB>
__global__ void __launch_bounds__(SUB ? 256 : F::V == 8 ? kFwdThreads : kFwdOddThreads, SUB ? (F::V == 8 ? 4 : 2) : 1)
layer_fwd_kernel(const NormArgs A) {
    using XT = typename F::XT;
    constexpr int MODE = F::MODE, V = F::V, NV = 8 / V;
    extern __shared__ __align__(16) ulonglong2 own[];
    ulonglong2 *wq = own, *bq = own + 2 * blockDim.x;
    RowSums<SUB> sums(A);
    const int tid = SUB ? threadIdx.x % A.tpr : threadIdx.x;
    const unsigned rows = SUB ? blockDim.x / A.tpr : 1, lane_row = SUB ? threadIdx.x / A.tpr : 0;
    const unsigned row0 = blockIdx.x / sums.K * rows;
    const Columns<MODE> c(A, sums.rank, tid, row0 + lane_row);
    const unsigned mine = own_columns(c);
    keep_columns<XT, MODE>(A.w_post, A.w32, 1.f, c, mine, wq);
    keep_columns<XT, MODE>(A.w_pre, A.w32, 0.f, c, mine, bq);
    const unsigned N = (unsigned)A.N, step = gridDim.x / sums.K * rows;
    Raw<XT, V> ry[NV] = {}, rr[NV] = {};
    auto fetch = [&](unsigned i) {
        if (i >= N) return;
        const RowAt at(A, i);
        const bool inside = i + 8 < N;  // the rows behind it hold a vector's columns past its end
        load8<XT, MODE>(ry, A.y, F::Y32, at.in(A, A.ys), c, inside);
        if constexpr (F::RES) load8<XT, MODE>(rr, A.residual, F::R32, at.in(A, A.rs), c, inside);
    };
    unsigned first = row0;
    fetch(first + lane_row);
    for (; first < N; first += step) {  // N + step + rows < 2^32
        const unsigned i = first + lane_row;
        const bool in = i < N;
        F2 r[4], w[4], b[4];
        trim8<XT, MODE>(ry, F::Y32, c);
        values8<XT, V>(ry, F::Y32, r);
        if constexpr (F::RES) {
            F2 t[4];
            trim8<XT, MODE>(rr, F::R32, c);
            values8<XT, V>(rr, F::R32, t);
#pragma unroll
            for (int v = 0; v < 4; ++v) r[v] = add2(r[v], t[v]);
            if (in) store8<XT, MODE>(A.r_out, F::R32, (long long)i * A.D, c, r);
            if constexpr (!F::R32) rounded<XT>(r);
        }
        fetch(i + step);  // the next row's values are on their way during this row's sums
        float s[1] = {sum8(r)};
        sums.template sum<1>(s);
        centre(r, mean_of(A, s[0]), mine, r);
        s[0] = dot8(r, r);
        own_read(wq, w);
        own_read(bq, b);
        sums.template sum<1>(s);
        const float rho = rsqrtf(fmaf(s[0], A.inv_d, A.eps));
#pragma unroll
        for (int v = 0; v < 4; ++v) r[v] = fma2(mul2(r[v], f2(rho)), w[v], b[v]);
        if (in) store8<XT, MODE>(A.n_out, false, (long long)i * A.D, c, r);
    }
    sums.end();
}

// dresidual: d r in r's type; dy: d r in the call's type (may be null)
template <class F, bool SUB>
__global__ void __launch_bounds__(SUB ? 256 : F::V == 8 ? kFwdThreads : kFwdOddThreads, SUB ? (F::MODE == kVec || !F::RES ? 4 : 2) : 1)
layer_bwd_kernel(const NormArgs A) {
    using XT = typename F::XT;
    constexpr int MODE = F::MODE, V = F::V, NV = 8 / V;
    extern __shared__ __align__(16) ulonglong2 own[];
    ulonglong2 *wq = own, *dq = own + 2 * blockDim.x, *bq = own + 4 * blockDim.x;
    RowSums<SUB> sums(A);
    const int tid = SUB ? threadIdx.x % A.tpr : threadIdx.x;
    const unsigned rows = SUB ? blockDim.x / A.tpr : 1, lane_row = SUB ? threadIdx.x / A.tpr : 0;
    const unsigned row0 = blockIdx.x / sums.K * rows;
    const Columns<MODE> c(A, sums.rank, tid, row0 + lane_row);
    const unsigned mine = own_columns(c);
    keep_columns<XT, MODE>(A.w_post, A.w32, 1.f, c, mine, wq);
    {
        const F2 zero[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
        own_write(dq, zero);
        own_write(bq, zero);
    }
    const unsigned N = (unsigned)A.N, step = gridDim.x / sums.K * rows;
    Raw<XT, V> rr[NV] = {}, rn[NV] = {}, rd[NV] = {};
    auto fetch = [&](unsigned i) {
        if (i >= N) return;
        const RowAt at(A, i);
        const bool inside = i + 8 < N;
        load8<XT, MODE>(rr, A.y, F::R32, at.in(A, A.ys), c, inside);
        load8<XT, MODE>(rn, A.dn, false, at.in(A, A.dns), c, inside);
        if constexpr (F::RES) load8<XT, MODE>(rd, A.dr, F::R32, at.in(A, A.drs), c, inside);
    };
    unsigned first = row0;
    fetch(first + lane_row);
    for (; first < N; first += step) {
        const unsigned i = first + lane_row;
        const bool in = i < N;
        const long long o = (long long)i * A.D;
        F2 u[4], m[4], e[4], w[4], acc[4];
        trim8<XT, MODE>(rr, F::R32, c);
        values8<XT, V>(rr, F::R32, u);
        trim8<XT, MODE>(rn, false, c);
        values8<XT, V>(rn, false, m);
        if constexpr (F::RES) {
            trim8<XT, MODE>(rd, F::R32, c);
            values8<XT, V>(rd, F::R32, e);
        }
        if (SUB && first + rows > N && !in) {  // the last turn's rows past the end count as 0
#pragma unroll
            for (int v = 0; v < 4; ++v) u[v] = m[v] = e[v] = f2(0.f);
        }
        fetch(i + step);  // the next row's values are on their way during this row's sums
        own_read(bq, acc);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = add2(acc[v], m[v]);
        own_write(bq, acc);
        own_read(wq, w);
        F2 dn[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) dn[v] = m[v], m[v] = mul2(m[v], w[v]);
        float s[2] = {sum8(u), sum8(m)};
        sums.template sum<2>(s);
        const float mean_m = mean_of(A, s[1]);
        centre(u, mean_of(A, s[0]), mine, u);
        s[0] = dot8(u, u), s[1] = dot8(m, u);
        sums.template sum<2>(s);
        const float rho = rsqrtf(fmaf(s[0], A.inv_d, A.eps)), k = s[1] * A.inv_d * rho * rho;
        own_read(dq, acc);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            acc[v] = fma2(mul2(dn[v], u[v]), f2(rho), acc[v]);
            const F2 t = mul2(fma2(u[v], f2(-k), add2(m[v], f2(-mean_m))), f2(rho));
            if constexpr (F::RES) e[v] = add2(e[v], t);
            else e[v] = t;
        }
        own_write(dq, acc);
        if (in) {
            store8<XT, MODE>(A.dresidual, F::R32, o, c, e);
            if (A.dy) store8<XT, MODE>(A.dy, F::Y32, o, c, e);
        }
    }
    sums.end();
    write_parts<XT, MODE, SUB>(A, c, dq, bq, rows, row0, sums.K);
}

}  // namespace norm
}  // namespace lattice

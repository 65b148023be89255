// block_norm.cuh -- the norm after a block with its gate and residual scale, joined with the
// norm before the next block, and the backward pass of both (sm_100a).
//
// Per row of D elements:
//   u = y rho1, rho1 = 1/sqrt(mean y^2 + eps)      (or u = y without the norm after)
//   v = scale u w_post act(gate)
//   r = residual + v                                (or r = v)
//   n = r rho2 w_pre, rho2 = 1/sqrt(mean r^2 + eps) (if wanted)
// Backward, from dr and dn:
//   e  = dr + rho2 (w_pre dn - r rho2^2 mean(w_pre dn r)),  d residual = e
//   dv = scale e,  d gate = dv u w_post act'(gate),  du = dv w_post act(gate)
//   dy = rho1 (du - y rho1^2 mean(du y))
//   dw_post = sum over rows of dv u act(gate),  dw_pre = sum over rows of dn r rho2
//
// HBM bounds both: every input is read once and every output written once, a row's values
// stay in registers between its reductions, and what is left is to keep enough rows in
// flight. A row of up to 256 elements takes a part of a warp (8 elements per thread) and its
// sums are shuffles; a longer one takes a CTA. CTAs stay and take rows by turns, so each
// thread keeps its columns' weights, and their gradients' sums, in registers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "args.h"

namespace lattice {
namespace norm {

constexpr int kNone = 0, kSigmoid = 1, kSilu = 2, kGelu = 3;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ uint32_t pack(__nv_bfloat16, float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t pack(__half, float a, float b) {
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void unpack(__nv_bfloat16, uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(__half, uint32_t w, float& a, float& b) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = t.x, b = t.y;
}

// V elements as read: fp32 or XT (f32 says which)
template <class XT, int V>
struct Raw {
    uint32_t w[V];
};
template <class XT, int V>
__device__ __forceinline__ Raw<XT, V> load(const void* p, bool f32, long long i) {
    Raw<XT, V> r;
    if constexpr (V == 1) {
        if (sizeof(XT) == 4 || f32) r.w[0] = static_cast<const uint32_t*>(p)[i];
        else r.w[0] = static_cast<const uint16_t*>(p)[i];
    } else {
        static_assert(V == 8, "vectors of 8");
        if (sizeof(XT) == 4 || f32) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
            const uint4 a = q[0], b = q[1];
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w, r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        }
    }
    return r;
}
template <class XT, int V>
__device__ __forceinline__ void values(const Raw<XT, V>& r, bool f32, float* f) {
    if (sizeof(XT) == 4 || f32) {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = __uint_as_float(r.w[v]);
    } else if constexpr (sizeof(XT) == 2) {
        if constexpr (V == 1) {
            float other;
            unpack(XT(), r.w[0], f[0], other);
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 2) unpack(XT(), r.w[v / 2], f[v], f[v + 1]);
        }
    }
}
template <class XT, int V>
__device__ __forceinline__ void store(void* p, bool f32, long long i, const float* f) {
    if constexpr (V == 1) {
        if (sizeof(XT) == 4 || f32) static_cast<float*>(p)[i] = f[0];
        else put(static_cast<XT*>(p) + i, f[0]);
    } else if (sizeof(XT) == 4 || f32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else if constexpr (sizeof(XT) == 2) {
        *reinterpret_cast<uint4*>(static_cast<XT*>(p) + i) =
            make_uint4(pack(XT(), f[0], f[1]), pack(XT(), f[2], f[3]), pack(XT(), f[4], f[5]), pack(XT(), f[6], f[7]));
    }
}

// The gate's activation and, if wanted, its derivative. The normal distribution function of
// gelu is formula 7.1.26 of Abramowitz and Stegun's Handbook (absolute error 7.5e-8 here),
// whose exponential the derivative needs too.
template <bool SLOPE>
__device__ __forceinline__ void activate(int act, float g, float& f, float& df) {
    if (act == kGelu) {
        const float x = fabsf(g) * 0.70710678f;
        const float e = exp2f(-0.72134752f * g * g);  // exp(-g^2/2)
        const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
        float p = 1.061405429f;
        p = fmaf(p, t, -1.453152027f);
        p = fmaf(p, t, 1.421413741f);
        p = fmaf(p, t, -0.284496736f);
        p = fmaf(p, t, 0.254829592f);
        const float tail = 0.5f * p * t * e;
        const float cdf = g >= 0.f ? 1.f - tail : tail;
        f = g * cdf;
        if constexpr (SLOPE) df = fmaf(g * 0.39894228f, e, cdf);
    } else {
        const float s = __fdividef(1.f, 1.f + __expf(-g));
        f = act == kSilu ? g * s : s;
        if constexpr (SLOPE) df = act == kSilu ? s * fmaf(g, 1.f - s, 1.f) : s * (1.f - s);
    }
}

// Sums of M values over the threads of a row: `tpr` lanes of a warp, or the CTA (red: two
// buffers by turns, so that one barrier per sum is enough).
template <bool CTA, int M>
__device__ __forceinline__ void row_sum(float* v, int tpr, float (*red)[32][M], int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (CTA || o < tpr)
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    if constexpr (CTA) {
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int m = 0; m < M; ++m) red[turn][warp][m] = v[m];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] = 0.f;
        for (int w = 0; w < nw; ++w)
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += red[turn][w][m];
    }
}

// Where row i of a strided array starts: groups of A.G rows, contiguous within a group.
__device__ __forceinline__ long long row_start(const NormArgs& A, long long stride, unsigned i, unsigned grp) {
    return (long long)grp * stride + (long long)(i - grp * A.G) * A.D;
}

template <class XT, bool CTA, int V, int NV>
__global__ void __launch_bounds__(CTA ? 1024 : 256) norm_fwd_kernel(const NormArgs A) {
    __shared__ float red1[2][32][1], red2[2][32][1];
    const int tpr = A.tpr, tid = CTA ? threadIdx.x : threadIdx.x % tpr;
    const int rows = CTA ? 1 : blockDim.x / tpr;  // per CTA and turn
    const int D = A.D;
    float wq[NV][V], wp[NV][V];  // the columns' weights
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + tid) * V;
        on[j] = c < D;
#pragma unroll
        for (int v = 0; v < V; ++v) wq[j][v] = A.scale, wp[j][v] = 1.f;
        if (on[j] && A.w_post) {
            values<XT, V>(load<XT, V>(A.w_post, A.w32, c), A.w32, wq[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) wq[j][v] *= A.scale;
        }
        if (on[j] && A.w_pre) values<XT, V>(load<XT, V>(A.w_pre, A.w32, c), A.w32, wp[j]);
    }
    int turn = 0;
    for (long long first = (long long)blockIdx.x * rows; first < A.N; first += (long long)gridDim.x * rows, turn ^= 1) {
        const long long i = first + (CTA ? 0 : threadIdx.x / tpr);
        const bool in = i < A.N;
        const unsigned grp = A.G == 1 ? (unsigned)i : (unsigned)i / A.G;
        const long long oy = row_start(A, A.ys, (unsigned)i, grp), og = row_start(A, A.gs, (unsigned)i, grp),
                        os = row_start(A, A.rs, (unsigned)i, grp), oo = i * D;
        Raw<XT, V> ry[NV], rg[NV], rr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + tid) * V;
            if (in && on[j]) {
                ry[j] = load<XT, V>(A.y, A.y32, oy + c);
                if (A.gate) rg[j] = load<XT, V>(A.gate, false, og + c);
                if (A.residual) rr[j] = load<XT, V>(A.residual, A.r32, os + c);
            }
        }
        float r[NV][V], s1[1] = {0.f}, s2[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            values<XT, V>(ry[j], A.y32, r[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!(in && on[j])) r[j][v] = 0.f;
                s1[0] = fmaf(r[j][v], r[j][v], s1[0]);
            }
        }
        float rho1 = 1.f;
        if (A.post) {
            row_sum<CTA, 1>(s1, tpr, red1, turn);
            rho1 = rsqrtf(fmaf(s1[0], A.inv_d, A.eps));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!(in && on[j])) continue;
            float g[V], res[V];
            if (A.gate) values<XT, V>(rg[j], false, g);
            if (A.residual) values<XT, V>(rr[j], A.r32, res);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float t = r[j][v] * rho1 * wq[j][v];
                if (A.gate) {
                    float f, df;
                    activate<false>(A.act, g[v], f, df);
                    t *= f;
                }
                r[j][v] = A.residual ? res[v] + t : t;
                s2[0] = fmaf(r[j][v], r[j][v], s2[0]);
            }
            store<XT, V>(A.r_out, A.o32, oo + (j * tpr + tid) * V, r[j]);
        }
        if (A.n_out) {
            row_sum<CTA, 1>(s2, tpr, red2, turn);
            const float rho2 = rsqrtf(fmaf(s2[0], A.inv_d, A.eps));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!(in && on[j])) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) r[j][v] = r[j][v] * rho2 * wp[j][v];
                store<XT, V>(A.n_out, false, oo + (j * tpr + tid) * V, r[j]);
            }
        }
    }
}

template <class XT, bool CTA, int V, int NV>
__global__ void __launch_bounds__(CTA && NV * V > 8 ? 512 : 256) norm_bwd_kernel(const NormArgs A) {
    __shared__ float red1[2][32][1], red2[2][32][2], red3[2][32][1];
    const int tpr = A.tpr, tid = CTA ? threadIdx.x : threadIdx.x % tpr;
    const int rows = CTA ? 1 : blockDim.x / tpr;
    const int D = A.D;
    const bool pre = A.dn != nullptr;
    float wq[NV][V], wp[NV][V], dq[NV][V], dp[NV][V];  // weights (w_post with the scale) and their gradients
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + tid) * V;
        on[j] = c < D;
#pragma unroll
        for (int v = 0; v < V; ++v) wq[j][v] = A.scale, wp[j][v] = 1.f, dq[j][v] = dp[j][v] = 0.f;
        if (on[j] && A.w_post) {
            values<XT, V>(load<XT, V>(A.w_post, A.w32, c), A.w32, wq[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) wq[j][v] *= A.scale;
        }
        if (on[j] && A.w_pre) values<XT, V>(load<XT, V>(A.w_pre, A.w32, c), A.w32, wp[j]);
    }
    int turn = 0;
    for (long long first = (long long)blockIdx.x * rows; first < A.N; first += (long long)gridDim.x * rows, turn ^= 1) {
        const long long i = first + (CTA ? 0 : threadIdx.x / tpr);
        const bool in = i < A.N;
        const unsigned grp = A.G == 1 ? (unsigned)i : (unsigned)i / A.G;
        const long long oy = row_start(A, A.ys, (unsigned)i, grp), og = row_start(A, A.gs, (unsigned)i, grp),
                        os = row_start(A, A.rs, (unsigned)i, grp), od = row_start(A, A.drs, (unsigned)i, grp),
                        on_ = row_start(A, A.dns, (unsigned)i, grp), oo = i * D;
        Raw<XT, V> ry[NV], rg[NV], rr[NV], rd[NV], rn[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + tid) * V;
            if (in && on[j]) {
                ry[j] = load<XT, V>(A.y, A.y32, oy + c);
                if (A.gate) rg[j] = load<XT, V>(A.gate, false, og + c);
                if (A.residual && pre) rr[j] = load<XT, V>(A.residual, A.r32, os + c);
                if (pre) rn[j] = load<XT, V>(A.dn, false, on_ + c);
                if (A.dr) rd[j] = load<XT, V>(A.dr, A.o32, od + c);
            }
        }
        float y[NV][V], e[NV][V], s1[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            values<XT, V>(ry[j], A.y32, y[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!(in && on[j])) y[j][v] = 0.f;
                s1[0] = fmaf(y[j][v], y[j][v], s1[0]);
            }
        }
        float rho1 = 1.f;
        if (A.post) {
            row_sum<CTA, 1>(s1, tpr, red1, turn);
            rho1 = rsqrtf(fmaf(s1[0], A.inv_d, A.eps));
        }
        float f[NV][V], df[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[V];
            if (A.gate) values<XT, V>(rg[j], false, g);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[j][v] = 1.f, df[j][v] = 0.f;
                if (A.gate) activate<true>(A.act, g[v], f[j][v], df[j][v]);
            }
            if (A.dr) values<XT, V>(rd[j], A.o32, e[j]);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) e[j][v] = 0.f;
        }
        if (pre) {
            float r[NV][V], dn[NV][V], s2[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float res[V];
                if (A.residual) values<XT, V>(rr[j], A.r32, res);
                values<XT, V>(rn[j], false, dn[j]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float t = y[j][v] * rho1 * wq[j][v] * f[j][v];
                    r[j][v] = A.residual ? res[v] + t : t;
                    if (!(in && on[j])) r[j][v] = dn[j][v] = 0.f;
                    s2[0] = fmaf(r[j][v], r[j][v], s2[0]);
                    s2[1] = fmaf(r[j][v], dn[j][v] * wp[j][v], s2[1]);
                }
            }
            row_sum<CTA, 2>(s2, tpr, red2, turn);
            const float rho2 = rsqrtf(fmaf(s2[0], A.inv_d, A.eps));
            const float k = rho2 * rho2 * rho2 * s2[1] * A.inv_d;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dp[j][v] = fmaf(dn[j][v], r[j][v] * rho2, dp[j][v]);
                    e[j][v] += rho2 * wp[j][v] * dn[j][v] - k * r[j][v];
                }
        }
        // e: d residual, then du without rho1
        float s3[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const long long o = oo + (j * tpr + tid) * V;
            if (!(in && on[j])) {
#pragma unroll
                for (int v = 0; v < V; ++v) e[j][v] = 0.f;
                continue;
            }
            if (A.dresidual) store<XT, V>(A.dresidual, A.r32, o, e[j]);
            float dg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = y[j][v] * rho1, t = e[j][v] * u;
                dg[v] = t * wq[j][v] * df[j][v];
                dq[j][v] = fmaf(t, f[j][v], dq[j][v]);
                e[j][v] *= wq[j][v] * f[j][v];
                s3[0] = fmaf(e[j][v], y[j][v], s3[0]);
            }
            if (A.dgate) store<XT, V>(A.dgate, false, o, dg);
        }
        float k = 0.f;
        if (A.post) {
            row_sum<CTA, 1>(s3, tpr, red3, turn);
            k = rho1 * rho1 * rho1 * s3[0] * A.inv_d;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!(in && on[j])) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) e[j][v] = e[j][v] * rho1 - k * y[j][v];
            store<XT, V>(A.dy, A.y32, oo + (j * tpr + tid) * V, e[j]);
        }
    }
    // the weights' gradients: the CTA's sums to its row of the workspace, added up by norm_dw_kernel
    if (!A.parts) return;
    if constexpr (CTA) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (j * tpr + tid) * V + v;
                if (c >= D) continue;
                float* p = A.parts + (long long)blockIdx.x * 2 * D + c;
                p[0] = dq[j][v];
                p[D] = dp[j][v];
            }
    } else {
        // rows of the CTA side by side: the first group's threads add them up, one by one
        __shared__ float side[256 * NV * V];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) side[(j * V + v) * 256 + threadIdx.x] = k ? dp[j][v] : dq[j][v];
            __syncthreads();
            if ((int)threadIdx.x < tpr)
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int c = (j * tpr + tid) * V + v;
                        float t = 0.f;
                        for (int q = 0; q < rows; ++q) t += side[(j * V + v) * 256 + q * tpr + tid];
                        if (c < D) A.parts[(long long)blockIdx.x * 2 * D + k * D + c] = t;
                    }
        }
    }
}

// dw = scale (w_post) or 1 (w_pre) times the column sums of [parts][2 D]: 32 columns and 8
// slices of the rows per CTA, slices added up in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* parts, int nparts, int D, float scale, float* dw_post,
                                                      float* dw_pre) {
    __shared__ float sum[8][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * D)
        for (int i = slice; i < nparts; i += 8) t += parts[(long long)i * 2 * D + c];
    sum[slice][lane] = t;
    __syncthreads();
    if (slice || c >= 2 * D) return;
    for (int s = 1; s < 8; ++s) t += sum[s][lane];
    if (c < D) {
        if (dw_post) dw_post[c] = t * scale;
    } else if (dw_pre) {
        dw_pre[c - D] = t;
    }
}

}  // namespace norm
}  // namespace lattice

// selective.cuh -- selective state space scan over whole sequences, its backward pass and its
// single-token step (sm_100a).
//
// Per (batch, channel e) with N states, dt = softplus(dt_raw + bias) (or as given):
//   h_t[n] = a_t[n] h_{t-1}[n] + dt_t x_t b_t[n],  a_t[n] = exp(dt_t A[e][n])
//   y_t = (sum_n c_t[n] h_t[n] + skip x_t) silu(z_t)
// b and c are shared by the channels of a group. Backward, with w = dy silu(z):
//   g_t[n] = w_t c_t[n] + a_{t+1}[n] g_{t+1}[n]
//   dc_t[n] = sum_e w_t h_t[n],  db_t[n] = sum_e g_t[n] dt_t x_t
//   q_t[n] = g_t[n] a_t[n] h_{t-1}[n],  dA[n] = sum_t q_t[n] dt_t,
//   du_t = sum_n g_t[n] b_t[n],  dx_t = dt_t du_t + skip w_t,  ddt_t = sum_n q_t[n] A[n] + x_t du_t
//
// What bounds it: N exponentials and some 4 N (backward 16 N) multiply-adds per element of x stand
// against a few bytes, so the CUDA cores do, not HBM. An SM sub-partition starts a warp's exponentials
// every 8.1 cycles, its multiply-adds every 1.1 (packed pairs: 2.2), its shuffles every 4.1 and its selects every
// 2 (measured); the layout keeps every state's work on those units at about the exponential's 8.
//
// Layout: a channel's states are split over L lanes, S (4 or 2) each, so a warp has 32/L channels and a
// CTA 8 warps. y's sum over n is a shuffle over L lanes, for four tokens at once (each lane
// hands half of its tokens on per step). What belongs to a channel and not to its states (softplus, dt x, the
// gate, the skip) is computed once per (token, channel) by the CTA, 16 tokens at a time, and passed on through
// shared memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "args.h"
#include "f32x2.cuh"

namespace lattice {
namespace selective {

constexpr int TT = kSelTile, NT = kSelThreads, NW = NT / 32;
constexpr unsigned ALL = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// Two neighbouring channels as read.
template <class T>
struct Pair {
    uint32_t w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Pair<T> load2(const void* base, long long i, int n, bool vec) {
    Pair<T> r;
    if constexpr (sizeof(T) == 4) {
        const uint32_t* p = static_cast<const uint32_t*>(base) + i;
        if (vec && n == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            r.w[0] = v.x, r.w[1] = v.y;
        } else {
            r.w[0] = n > 0 ? p[0] : 0u;
            r.w[1] = n > 1 ? p[1] : 0u;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        if (vec && n == 2) {
            r.w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            r.w[0] = n > 0 ? p[0] : 0u;
            if (n > 1) r.w[0] |= (uint32_t)p[1] << 16;
        }
    }
    return r;
}
template <class T>
__device__ __forceinline__ F2 value2(const Pair<T>& r) {
    if constexpr (sizeof(T) == 4) {
        return f2(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]));
    } else if constexpr (std::is_same<T, __half>::value) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r.w[0]));
        return f2(v.x, v.y);
    } else {
        return f2(__uint_as_float(r.w[0] << 16), __uint_as_float(r.w[0] & 0xffff0000u));
    }
}
template <class T>
__device__ __forceinline__ void store2(void* base, long long i, F2 v, int n, bool vec) {
    float a, b;
    parts(v, a, b);
    T* p = static_cast<T*>(base) + i;
    if (vec && n == 2) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float2*>(p) = make_float2(a, b);
        } else if constexpr (std::is_same<T, __half>::value) {
            *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
        } else {
            *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
        }
        return;
    }
    if (n > 0) put(p, a);
    if (n > 1) put(p + 1, b);
}
// dt: fp32 or XT
template <class XT>
__device__ __forceinline__ Pair<float> load_dt(const SelArgs& A, long long i, int n) {
    if (sizeof(XT) == 4 || A.dt32) return load2<float>(A.dt, i, n, A.vec);
    const Pair<XT> p = load2<XT>(A.dt, i, n, A.vec);
    Pair<float> r;
    r.w[0] = p.w[0], r.w[1] = 0u;
    return r;
}
template <class XT>
__device__ __forceinline__ F2 value_dt(const SelArgs& A, const Pair<float>& r) {
    if constexpr (sizeof(XT) == 2) {
        if (!A.dt32) {
            Pair<XT> p;
            p.w[0] = r.w[0];
            return value2(p);
        }
    }
    return value2(r);
}

// exp(dt A) of two states, t = dt A log2(e). The approximate exponential's errors near 1 are not centred (mean
// -2e-8 for t in [-1/2, -2^-8], measured), and a retention of R steps multiplies a mean error by R.
// So -0.36 <= t <= 0 takes 1 + t q(t) instead, a minimax polynomial (1.6e-8, and 0 at t = 0) whose
// last step rounds to nearest; below, R is at most 4. The integer comparison holds for negative t alone.
constexpr float kNear = -0.36f;
__device__ __forceinline__ F2 decay(F2 t) {
    F2 p = fma2(f2(0.008524463512003422f), t, f2(0.055181119590997696f));
    p = fma2(p, t, f2(0.24018850922584534f));
    p = fma2(p, t, f2(0.6931458115577698f));
    p = fma2(p, t, f2(1.f));
    float t0, t1, p0, p1;
    parts(t, t0, t1), parts(p, p0, p1);
    const float e0 = ex2(t0), e1 = ex2(t1);
    const int near = __float_as_int(kNear);
    return f2(__float_as_int(t0) <= near ? p0 : e0, __float_as_int(t1) <= near ? p1 : e1);
}

// softplus(v) = max(v, 0) + log(1 + t), t = exp(-|v|), and its slope 1/(1 + exp(-v)). log(1 + t)/t is a
// polynomial of degree 9 (minimax on [0, 1], relative error 5e-9), so small steps keep their relative accuracy.
__device__ __forceinline__ F2 softplus(F2 v, F2* slope) {
    const F2 t = each(v, [](float a) { return ex2(-fabsf(a) * kLog2e); });
    F2 p = fma2(f2(-0.003244034f), t, f2(0.019851461f));
    p = fma2(p, t, f2(-0.05695953f));
    p = fma2(p, t, f2(0.10603654f));
    p = fma2(p, t, f2(-0.15305592f));
    p = fma2(p, t, f2(0.19675939f));
    p = fma2(p, t, f2(-0.24954134f));
    p = fma2(p, t, f2(0.33329964f));
    p = fma2(p, t, f2(-0.49999902f));
    p = fma2(p, t, f2(1.f));
    if (slope) {
        const F2 r = each(add2(t, f2(1.f)), rcp), s = mul2(t, r);
        float v0, v1, r0, r1, s0, s1;
        parts(v, v0, v1), parts(r, r0, r1), parts(s, s0, s1);
        *slope = f2(v0 >= 0.f ? r0 : s0, v1 >= 0.f ? r1 : s1);
    }
    return fma2(p, t, each(v, [](float a) { return max_nan(a, 0.f); }));
}
// 1/(1 + exp(-z))
__device__ __forceinline__ F2 sigmoid(F2 z) {
    return each(each(mul2(z, f2(-kLog2e)), [](float n) { return 1.f + ex2(n); }), rcp);
}
// dt of two channels from what was read
template <class XT>
__device__ __forceinline__ F2 step_size(const SelArgs& A, const Pair<float>& raw, F2 bias, F2* slope) {
    const F2 v = add2(value_dt<XT>(A, raw), bias);
    if (A.softplus) return softplus(v, slope);
    if (slope) *slope = f2(1.f);
    return v;
}
__device__ __forceinline__ F2 low(ulonglong2 v) { return F2{v.x}; }
__device__ __forceinline__ F2 high(ulonglong2 v) { return F2{v.y}; }
__device__ __forceinline__ ulonglong2 both(F2 a, F2 b) { return make_ulonglong2(a.v, b.v); }
__device__ __forceinline__ float total(F2 a) {
    float x, y;
    parts(a, x, y);
    return x + y;
}
__device__ __forceinline__ float total(F2 a, F2 b) { return total(add2(a, b)); }

// v0 and v1 summed over two lanes that differ in `bit`: the lane without it keeps v0's sum.
__device__ __forceinline__ float halve(float v0, float v1, int lane, int bit) {
    const bool up = lane & bit;
    const float keep = up ? v1 : v0, give = up ? v0 : v1;
    return keep + __shfl_xor_sync(ALL, give, bit);
}

// Where a CTA works: a tile of CT channels of one group, one sequence, one segment of the time axis.
template <int L>
struct Place {
    static constexpr int CH = 32 / L, CT = NW * CH, PAIRS = CT / 2, ROWS = NT / PAIRS;
    static constexpr int PI = (TT + ROWS - 1) / ROWS;  // pairs per thread of a tile of tokens
    static constexpr int CTP = CT + 8;                 // floats of a row of sums, rows apart in the banks
    int b, s, ct, g, c0, cend, t0, t1, te;             // tokens t0..t1, te: up to the sequence's end
    int lane, gl, cl, c, ch, cp, row;                  // states' lane, channel; the pair and first row of the thread
    bool live;
    __device__ __forceinline__ Place(const SelArgs& A) {
        const int nt = A.G * A.tiles;
        unsigned blk = blockIdx.x;
        ct = blk % nt, blk /= nt;
        s = blk % A.nseg, b = blk / A.nseg;
        g = ct / A.tiles, c0 = g * A.Eg + (ct - g * A.tiles) * CT, cend = (g + 1) * A.Eg;
        const int len = A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
        t0 = s * A.seg, t1 = min(A.T, t0 + A.seg), te = max(t0, min(t1, len));
        lane = threadIdx.x & 31, gl = lane % L, cl = lane / L, c = (threadIdx.x >> 5) * CH + cl, ch = c0 + c;
        live = ch < cend;
        cp = threadIdx.x % PAIRS, row = threadIdx.x / PAIRS;
    }
    __device__ __forceinline__ int pair() const { return c0 + 2 * cp; }
    __device__ __forceinline__ int width() const { return min(2, max(0, cend - pair())); }  // channels of the pair
    __device__ __forceinline__ long long seq() const { return b; }
};

// S states of a channel, of p[N]; 0 past N
template <int S>
__device__ __forceinline__ void load_states(const float* p, int n0, int N, bool vec, float* v) {
    if (S == 4 && vec) {
        if (n0 < N) {
            const float4 t = *reinterpret_cast<const float4*>(p + n0);
            v[0] = t.x, v[1] = t.y, v[S - 2] = t.z, v[S - 1] = t.w;
        } else {
#pragma unroll
            for (int k = 0; k < S; ++k) v[k] = 0.f;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = n0 + k < N ? p[n0 + k] : 0.f;
}
template <int S>
__device__ __forceinline__ void store_states(float* p, int n0, int N, bool vec, const float* v) {
    if (S == 4 && vec) {
        if (n0 < N) *reinterpret_cast<float4*>(p + n0) = make_float4(v[0], v[1], v[S - 2], v[S - 1]);
        return;
    }
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (n0 + k < N) p[n0 + k] = v[k];
}
template <int S>
__device__ __forceinline__ void pack(const float* v, F2* h) {
#pragma unroll
    for (int k = 0; k < S / 2; ++k) h[k] = f2(v[2 * k], v[2 * k + 1]);
}
template <int S>
__device__ __forceinline__ void unpack(const F2* h, float* v) {
#pragma unroll
    for (int k = 0; k < S / 2; ++k) parts(h[k], v[2 * k], v[2 * k + 1]);
}
// S states' values of b or c in shared memory
template <int S>
__device__ __forceinline__ void read_vec(const float* p, F2* v) {
    if constexpr (S == 4) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p);
        v[0].v = t.x, v[S / 2 - 1].v = t.y;
    } else {
        v[0].v = *reinterpret_cast<const unsigned long long*>(p);
    }
}
// A tile's rows of b or c: NB elements of [TT][NP] per thread.
template <int NP>
struct Rows {
    static constexpr int NB = (TT * NP + NT - 1) / NT;
};
template <class XT, int NP>
__device__ __forceinline__ void fetch_rows(const void* base, long long at, long long ts, int tb, int te, int N, XT* r) {
#pragma unroll
    for (int k = 0; k < Rows<NP>::NB; ++k) {
        const int i = threadIdx.x + k * NT, t = i / NP, n = i % NP;
        XT v = XT();
        if (t < TT && tb + t < te && n < N) v = static_cast<const XT*>(base)[at + (tb + t) * ts + n];
        r[k] = v;
    }
}

// ---- forward: all tokens of a segment, from the state that enters it
template <class XT, int L, int S>
struct FwdShared {
    static constexpr int NP = L * S, CT = Place<L>::CT, CTP = Place<L>::CTP;
    ulonglong2 dtu[TT * CT];  // (dt, dt, u, u), u = dt x
    float b[TT * NP], c[TT * NP];
    float y[TT * CTP];
};

template <class XT, int L, int S>
__global__ void __launch_bounds__(NT, 2) fwd_kernel(const SelArgs A) {
    using P = Place<L>;
    constexpr int NP = L * S, CT = P::CT, CTP = P::CTP, PI = P::PI, NB = Rows<NP>::NB, H = S / 2;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    FwdShared<XT, L, S>& sh = *reinterpret_cast<FwdShared<XT, L, S>*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * S, pw = p.width();
    F2 h[H], A2[H], bias = f2(0.f), skip = f2(0.f);
    {
        float v[S] = {};
        if (p.live) load_states<S>(A.A + (long long)p.ch * A.N, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] *= kLog2e;
        pack<S>(v, A2);
        const float* from = A.nseg > 1 ? A.seg_state + ((long long)(p.b * A.nseg + p.s) * A.E) * A.N
                            : A.h0   ? A.h0 + (long long)p.b * A.E * A.N
                                     : nullptr;
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] = 0.f;
        if (from && p.live) load_states<S>(from + (long long)p.ch * A.N, n0, A.N, A.vec_n, v);
        pack<S>(v, h);
        if (A.dt_bias) bias = value2(load2<float>(A.dt_bias, p.pair(), pw, false));
        if (A.skip) skip = value2(load2<float>(A.skip, p.pair(), pw, false));
    }
    const long long xat = p.b * A.xbs + p.pair(), dat = p.b * A.dbs + p.pair(), zat = p.b * A.zbs + p.pair(),
                    bat = p.b * A.bbs + p.g * A.N, cat = p.b * A.cbs + p.g * A.N, yat = (long long)p.b * A.T * A.E + p.pair();
    Pair<XT> rx[PI], rz[PI], kx[PI], kz[PI];
    Pair<float> rd[PI];
    XT rb[NB], rc[NB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load2<XT>(A.x, xat + t * A.xts, n, A.vec);
            rd[k] = load_dt<XT>(A, dat + t * A.dts, n);
            if (A.z) rz[k] = load2<XT>(A.z, zat + t * A.zts, n, A.vec);
        }
        fetch_rows<XT, NP>(A.b, bat, A.bts, tb, p.te, A.N, rb);
        fetch_rows<XT, NP>(A.c, cat, A.cts, tb, p.te, A.N, rc);
    };
    auto finish = [&](int tb) {  // the tile's outputs
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r;
            if (r >= TT || t >= p.te) continue;
            F2 y = *reinterpret_cast<const F2*>(sh.y + r * CTP + 2 * p.cp);
            y = fma2(skip, value2(kx[k]), y);
            if (A.z) {
                const F2 z = value2(kz[k]);
                y = mul2(y, mul2(z, sigmoid(z)));
            }
            store2<XT>(A.y, yat + (long long)t * A.E, y, pw, A.vec);
        }
    };
    if (p.t0 < p.te) fetch(p.t0);
    for (int tb = p.t0; tb < p.te; tb += TT) {
        __syncthreads();
        if (tb > p.t0 && A.y) finish(tb - TT);
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (r >= TT) continue;
            F2 dt = f2(0.f), u = f2(0.f);
            if (tb + r < p.te) {
                dt = step_size<XT>(A, rd[k], bias, nullptr);
                u = mul2(dt, value2(rx[k]));
            }
            kx[k] = rx[k], kz[k] = rz[k];
            float d0, d1, u0, u1;
            parts(dt, d0, d1), parts(u, u0, u1);
            sh.dtu[r * CT + 2 * p.cp] = both(f2(d0), f2(u0));
            sh.dtu[r * CT + 2 * p.cp + 1] = both(f2(d1), f2(u1));
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i < TT * NP) sh.b[i] = to_f(rb[k]), sh.c[i] = to_f(rc[k]);
        }
        if (tb + TT < p.te) fetch(tb + TT);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < TT; q += 4) {
            if (q % kSelMark == 0 && A.marks && tb + q < p.te && p.live) {
                float v[S];
                unpack<S>(h, v);
                store_states<S>(A.marks + (((long long)p.b * A.nmarks + (tb + q) / kSelMark) * A.E + p.ch) * A.N, n0, A.N, A.vec_n, v);
            }
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = q + j;
                const ulonglong2 du = sh.dtu[t * CT + p.c];
                F2 bv[H], cv[H];
                read_vec<S>(sh.b + t * NP + n0, bv);
                read_vec<S>(sh.c + t * NP + n0, cv);
                F2 yy;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    h[k] = fma2(decay(mul2(low(du), A2[k])), h[k], mul2(high(du), bv[k]));
                    yy = k ? fma2(h[k], cv[k], yy) : mul2(h[k], cv[k]);
                }
                y[j] = total(yy);
            }
            const float y01 = halve(y[0], y[1], p.lane, 1), y23 = halve(y[2], y[3], p.lane, 1);
            if constexpr (L == 2) {
                sh.y[(q + p.gl) * CTP + p.c] = y01;
                sh.y[(q + 2 + p.gl) * CTP + p.c] = y23;
            } else {
                float v = halve(y01, y23, p.lane, 2);
#pragma unroll
                for (int o = 4; o < L; o *= 2) v += __shfl_xor_sync(ALL, v, o);
                if (p.gl < 4) sh.y[(q + p.gl) * CTP + p.c] = v;
            }
        }
    }
    if (A.y) {
        __syncthreads();
        if (p.t0 < p.te) finish((p.te - 1 - p.t0) / TT * TT + p.t0);
        for (int t = p.te + p.row; t < p.t1; t += P::ROWS)  // behind the sequence's end
            store2<XT>(A.y, yat + (long long)t * A.E, f2(0.f), pw, A.vec);
    }
    if (A.h_out && p.s == A.nseg - 1 && p.live) {
        float v[S];
        unpack<S>(h, v);
        store_states<S>(A.h_out + ((long long)p.b * A.E + p.ch) * A.N, n0, A.N, A.vec_n, v);
    }
}

// ---- a segment's state from 0 at its end (REV: the cotangent from 0 at its start) and the sum of its dt
template <class XT, int L, int S>
struct SegShared {
    static constexpr int NP = L * S, CT = Place<L>::CT;
    ulonglong2 dtu[TT * CT];  // (dt, dt, w, w), w = dt x or dy silu(z)
    float v[TT * NP];         // b or c
    float2 sum[NT];
};

template <class XT, int L, int S, bool REV>
__global__ void __launch_bounds__(NT, 2) seg_kernel(const SelArgs A) {
    using P = Place<L>;
    constexpr int NP = L * S, CT = P::CT, PI = P::PI, NB = Rows<NP>::NB, H = S / 2;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    SegShared<XT, L, S>& sh = *reinterpret_cast<SegShared<XT, L, S>*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * S, pw = p.width();
    F2 h[H], A2[H], bias = f2(0.f), sum = f2(0.f);
    {
        float v[S] = {};
        if (p.live) load_states<S>(A.A + (long long)p.ch * A.N, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] *= kLog2e;
        pack<S>(v, A2);
#pragma unroll
        for (int k = 0; k < H; ++k) h[k] = f2(0.f);
        if (A.dt_bias) bias = value2(load2<float>(A.dt_bias, p.pair(), pw, false));
    }
    const void *src = REV ? A.dy : A.x, *vec = REV ? A.c : A.b;
    const long long sts = REV ? A.yts : A.xts, sat = p.b * (REV ? A.ybs : A.xbs) + p.pair(), dat = p.b * A.dbs + p.pair(),
                    zat = p.b * A.zbs + p.pair(), vts = REV ? A.cts : A.bts, vat = p.b * (REV ? A.cbs : A.bbs) + p.g * A.N;
    const bool gated = REV && A.z;
    Pair<XT> rx[PI], rz[PI];
    Pair<float> rd[PI];
    XT rv[NB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load2<XT>(src, sat + t * sts, n, A.vec);
            rd[k] = load_dt<XT>(A, dat + t * A.dts, n);
            if (gated) rz[k] = load2<XT>(A.z, zat + t * A.zts, n, A.vec);
        }
        fetch_rows<XT, NP>(vec, vat, vts, tb, p.te, A.N, rv);
    };
    const int tiles = (p.te - p.t0 + TT - 1) / TT;
    auto base = [&](int i) { return p.t0 + (REV ? tiles - 1 - i : i) * TT; };
    if (tiles) fetch(base(0));
    for (int i = 0; i < tiles; ++i) {
        const int tb = base(i);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (r >= TT) continue;
            F2 dt = f2(0.f), w = f2(0.f);
            if (tb + r < p.te) {
                dt = step_size<XT>(A, rd[k], bias, nullptr);
                w = value2(rx[k]);
                if constexpr (!REV) {
                    w = mul2(w, dt);
                } else if (gated) {
                    const F2 z = value2(rz[k]);
                    w = mul2(w, mul2(z, sigmoid(z)));
                }
            }
            sum = add2(sum, dt);
            float d0, d1, w0, w1;
            parts(dt, d0, d1), parts(w, w0, w1);
            sh.dtu[r * CT + 2 * p.cp] = both(f2(d0), f2(w0));
            sh.dtu[r * CT + 2 * p.cp + 1] = both(f2(d1), f2(w1));
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int j = threadIdx.x + k * NT;
            if (j < TT * NP) sh.v[j] = to_f(rv[k]);
        }
        if (i + 1 < tiles) fetch(base(i + 1));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int t = REV ? TT - 1 - j : j;
            const ulonglong2 du = sh.dtu[t * CT + p.c];
            F2 v[H];
            read_vec<S>(sh.v + t * NP + n0, v);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const F2 a = decay(mul2(low(du), A2[k]));
                if constexpr (REV) h[k] = mul2(a, fma2(high(du), v[k], h[k]));
                else h[k] = fma2(a, h[k], mul2(high(du), v[k]));
            }
        }
    }
    const long long at = (long long)(p.b * A.nseg + p.s) * A.E;
    if (p.live) {
        float v[S];
        unpack<S>(h, v);
        store_states<S>(A.seg_state + (at + p.ch) * A.N, n0, A.N, A.vec_n, v);
    }
    float s0, s1;
    parts(sum, s0, s1);
    sh.sum[threadIdx.x] = make_float2(s0, s1);
    __syncthreads();
    if (p.row == 0) {  // row by row, in order
        for (int r = 1; r < P::ROWS; ++r) {
            const float2 o = sh.sum[r * P::PAIRS + p.cp];
            s0 += o.x, s1 += o.y;
        }
        if (pw > 0) A.seg_sum[at + p.pair()] = s0;
        if (pw > 1) A.seg_sum[at + p.pair() + 1] = s1;
    }
}

// The states that enter the segments (REV: the cotangents that enter them from behind), in place.
template <bool REV>
__global__ void __launch_bounds__(256) join_kernel(const SelArgs A) {
    const long long per = (long long)A.E * A.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * A.B) return;
    const long long b = i / per, en = i - b * per, e = en / A.N;
    const float a = A.A[en] * kLog2e;
    const float* first = REV ? A.dh_T : A.h0;
    float h = first ? first[i] : 0.f;
    for (int k = 0; k < A.nseg; ++k) {
        const long long at = b * A.nseg + (REV ? A.nseg - 1 - k : k);
        float* p = A.seg_state + at * per + en;
        const float own = *p, keep = exp2f(a * A.seg_sum[at * A.E + e]);
        *p = h;
        h = fmaf(keep, h, own);
    }
}

// ---- one token: 4 states per thread, L lanes per channel
template <class XT, int L>
__global__ void __launch_bounds__(256) step_kernel(const SelArgs A) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = A.E;
    const long long bc = i / L;
    const int gl = (int)(i % L), n0 = gl * 4;
    const bool live = bc < per * A.B;
    const long long b = live ? bc / per : 0;
    const int e = live ? (int)(bc - b * per) : 0, g = e / A.Eg;
    float h[4] = {}, a[4] = {}, bv[4] = {}, cv[4] = {};
    float x = 0.f, dt = 0.f;
    if (live) {
        load_states<4>(A.h0 + (b * A.E + e) * A.N, n0, A.N, A.vec_n, h);
        load_states<4>(A.A + (long long)e * A.N, n0, A.N, A.vec_n, a);
        const XT *pb = static_cast<const XT*>(A.b) + b * A.bbs + g * A.N, *pc = static_cast<const XT*>(A.c) + b * A.cbs + g * A.N;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < A.N) bv[k] = to_f(pb[n0 + k]), cv[k] = to_f(pc[n0 + k]);
        x = to_f(static_cast<const XT*>(A.x)[b * A.xbs + e]);
        const long long di = b * A.dbs + e;
        dt = sizeof(XT) == 4 || A.dt32 ? static_cast<const float*>(A.dt)[di] : to_f(static_cast<const XT*>(A.dt)[di]);
        if (A.dt_bias) dt += A.dt_bias[e];
        if (A.softplus) {
            float other;
            parts(softplus(f2(dt), nullptr), dt, other);
        }
    }
    const float u = dt * x;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        float a0, a1;
        parts(decay(mul2(f2(dt * kLog2e), f2(a[k], a[k + 1]))), a0, a1);
        h[k] = fmaf(a0, h[k], u * bv[k]);
        h[k + 1] = fmaf(a1, h[k + 1], u * bv[k + 1]);
        y = fmaf(h[k], cv[k], fmaf(h[k + 1], cv[k + 1], y));
    }
#pragma unroll
    for (int o = 1; o < L; o *= 2) y += __shfl_xor_sync(ALL, y, o);
    if (!live) return;
    store_states<4>(A.h_out + (b * A.E + e) * A.N, n0, A.N, A.vec_n, h);
    if (gl) return;
    if (A.skip) y = fmaf(A.skip[e], x, y);
    if (A.z) {
        const float z = to_f(static_cast<const XT*>(A.z)[b * A.zbs + e]);
        y *= z * rcp(1.f + ex2(-z * kLog2e));
    }
    put(static_cast<XT*>(A.y) + b * A.E + e, y);
}

}  // namespace selective
}  // namespace lattice

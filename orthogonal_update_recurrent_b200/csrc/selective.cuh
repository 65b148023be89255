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
// Mid-size layer (8 x 4096 tokens of 2048 bf16 channels, 16 states, gate): 640 us with the backward pass's marks (614 us without),
// 1.7e12 states per second, 0.37 of the rate of the exponentials alone. A token costs a warp 48 instructions for 128 states, its share of the
// staging included, 58 % of the issue slots at 3.5 warps per scheduler; shared memory returns data 58 % of the time, the exponentials' units are
// busy 46 %, and a warp's own latencies fill the rest. One sequence of 65536 tokens of 1024 channels: 545 us, and 390 us for its 18
// segments' states (seg_kernel).
// One token of 256 sequences of 4096 channels, 137 MB of states: 27 us (step_kernel; reads and writes bind).
//
// Tried: two channels per lane, which share what is read of b and c, on half the threads (694 us; backward 1590 us, as fast as
// one); steps and inputs in shared memory twice, as the packed instructions take them (706 us); b and c there as 16 bits (slower).
//
// Layout: a channel's states are split over L lanes, S (4 or 2) each, so a warp has 32/L channels and a
// CTA 8 warps (2 for few channels). The lanes' parts of y's sum over n stand side by side in shared memory until the
// thread that finishes a token's channels adds them up. What belongs to a channel and not to its states (softplus, dt x, the
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

constexpr int TT = kSelTile;
constexpr unsigned ALL = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// V neighbouring channels (1, 2 or 4) as read, of type T
template <class T, int V>
struct Raw {
    static constexpr int W = sizeof(T) * V < 4 ? 1 : sizeof(T) * V / 4;
    uint32_t w[W];
};
template <class T, int V>
__device__ __forceinline__ Raw<T, V> none() {
    Raw<T, V> r;
#pragma unroll
    for (int k = 0; k < Raw<T, V>::W; ++k) r.w[k] = 0u;
    return r;
}
// n of them at p. VEC: n is 0 or V, and they can be read at once
template <bool VEC, class T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* p, int n) {
    Raw<T, V> r = none<T, V>();
    if constexpr (VEC && V > 1) {
        constexpr int W = Raw<T, V>::W;
        if (n > 0) {
            if constexpr (W == 4) {
                const uint4 t = *reinterpret_cast<const uint4*>(p);
                r.w[0] = t.x, r.w[W / 4] = t.y, r.w[W / 2] = t.z, r.w[W - 1] = t.w;
            } else if constexpr (W == 2) {
                const uint2 t = *reinterpret_cast<const uint2*>(p);
                r.w[0] = t.x, r.w[W - 1] = t.y;
            } else {
                r.w[0] = *reinterpret_cast<const uint32_t*>(p);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v >= n) continue;
            if constexpr (sizeof(T) == 4) r.w[v] = reinterpret_cast<const uint32_t*>(p)[v];
            else r.w[v / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[v] << (16 * (v & 1));
        }
    }
    return r;
}
// pairs of their values; a single one has 0 beside it
template <class T, int V>
__device__ __forceinline__ void values(const Raw<T, V>& r, F2* f) {
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) {
        if constexpr (sizeof(T) == 4) {
            f[k] = f2(__uint_as_float(r.w[2 * k]), V > 1 ? __uint_as_float(r.w[V > 1 ? 2 * k + 1 : 0]) : 0.f);
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r.w[k]));
            f[k] = f2(v.x, v.y);
        } else {
            f[k] = f2(__uint_as_float(r.w[k] << 16), __uint_as_float(r.w[k] & 0xffff0000u));
        }
    }
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 t = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&t);
    } else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&t);
    }
}
template <bool VEC, class T, int V>
__device__ __forceinline__ void store(T* p, const F2* f, int n) {
    float v[V + 1];
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) parts(f[k], v[2 * k], v[2 * k + 1]);
    if constexpr (VEC && V > 1) {
        if (n <= 0) return;
        if constexpr (sizeof(T) == 4) {
            if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[V - 2], v[V - 1]);
            else *reinterpret_cast<float2*>(p) = make_float2(v[0], v[V - 1]);
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[V - 2], v[V - 1]));
        } else {
            *reinterpret_cast<uint32_t*>(p) = pack2<T>(v[0], v[1]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n) put(p + k, v[k]);
    }
}
// Column c of token t of an array whose tokens are `ts` elements apart, from p on (the same for the whole CTA). VEC calls' arrays
// are less than 2^31 bytes from the first to the last token, so that 32-bit offsets do.
template <bool VEC, class T>
__device__ __forceinline__ T* token(T* p, int c, int t, long long ts) {
    if constexpr (VEC) return reinterpret_cast<T*>(reinterpret_cast<unsigned long long>(p) + ((unsigned)t * (unsigned)ts + (unsigned)c) * (unsigned)sizeof(T));
    else return p + (t * ts + c);
}
// V channels of dt, which are fp32 or XT
template <bool VEC, class XT, int V>
__device__ __forceinline__ Raw<float, V> load_dt(const SelArgs& A, const void* p, int c, int t, int n) {
    if (sizeof(XT) == 4 || A.dt32) return load<VEC, float, V>(token<VEC>(static_cast<const float*>(p), c, t, A.dts), n);
    const Raw<XT, V> v = load<VEC, XT, V>(token<VEC>(static_cast<const XT*>(p), c, t, A.dts), n);
    Raw<float, V> r = none<float, V>();
#pragma unroll
    for (int k = 0; k < Raw<XT, V>::W; ++k) r.w[k] = v.w[k];
    return r;
}
template <class XT, int V>
__device__ __forceinline__ void values_dt(const SelArgs& A, const Raw<float, V>& r, F2* f) {
    if constexpr (sizeof(XT) == 2) {
        if (!A.dt32) {
            Raw<XT, V> p;
#pragma unroll
            for (int k = 0; k < Raw<XT, V>::W; ++k) p.w[k] = r.w[k];
            values<XT, V>(p, f);
            return;
        }
    }
    values<float, V>(r, f);
}
// where dt's entries of sequence b begin
template <class XT>
__device__ __forceinline__ const void* dt_at(const SelArgs& A, int b) {
    return sizeof(XT) == 4 || A.dt32 ? static_cast<const void*>(static_cast<const float*>(A.dt) + b * A.dbs)
                                     : static_cast<const void*>(static_cast<const XT*>(A.dt) + b * A.dbs);
}

// exp(dt A) of two states, t = dt A log2(e). The approximate exponential's errors near 1 are not centred (mean
// -2e-8 for t in [-1/2, -2^-8], measured), and a retention of R steps multiplies a mean error by R.
// So -0.09 <= t <= 0 takes 1 + t q(t) instead, a minimax polynomial (6.7e-9, 1e-11 on the mean, and 0 at
// t = 0) whose last step rounds to nearest; below, R is at most 16. The integer comparison holds for negative t alone.
constexpr float kNear = -0.09f;
// of M pairs, step by step, so that no step waits for the one before it
template <int M>
__device__ __forceinline__ void decay(F2* t) {
    F2 p[M];
    float e[2 * M];
#pragma unroll
    for (int i = 0; i < M; ++i) p[i] = fma2(f2(0.053866468369960785f), t[i], f2(0.24014140665531158f));
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float t0, t1;
        parts(t[i], t0, t1);
        e[2 * i] = ex2(t0), e[2 * i + 1] = ex2(t1);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) p[i] = fma2(p[i], t[i], f2(0.6931459307670593f));
#pragma unroll
    for (int i = 0; i < M; ++i) p[i] = fma2(p[i], t[i], f2(1.f));
    const int near = __float_as_int(kNear);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float t0, t1, p0, p1;
        parts(t[i], t0, t1), parts(p[i], p0, p1);
        t[i] = f2(__float_as_int(t0) <= near ? p0 : e[2 * i], __float_as_int(t1) <= near ? p1 : e[2 * i + 1]);
    }
}
__device__ __forceinline__ F2 decay(F2 t) {
    decay<1>(&t);
    return t;
}

// softplus(v) = max(v, 0) + log(1 + t), t = exp(-|v|), and its slope 1/(1 + exp(-v)). log(1 + t)/t is a
// polynomial of degree 9 (minimax on [0, 1] with 1 at t = 0, rounded one coefficient after the other and refitted: relative error 5.3e-9,
// mean 6e-11), so small steps keep their relative accuracy.
__device__ __forceinline__ F2 softplus(F2 v, F2* slope) {
    const F2 t = each(v, [](float a) { return ex2(-fabsf(a) * kLog2e); });
    F2 p = fma2(f2(-0.0032910742f), t, f2(0.02008846f));
    p = fma2(p, t, f2(-0.057460483f));
    p = fma2(p, t, f2(0.10661371f));
    p = fma2(p, t, f2(-0.15344977f));
    p = fma2(p, t, f2(0.19692121f));
    p = fma2(p, t, f2(-0.2495802f));
    p = fma2(p, t, f2(0.33330464f));
    p = fma2(p, t, f2(-0.4999993f));
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
// dt of V channels from what was read
template <class XT, int V>
__device__ __forceinline__ void step_sizes(const SelArgs& A, const Raw<float, V>& raw, const F2* bias, F2* dt, F2* slope) {
    values_dt<XT, V>(A, raw, dt);
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) {
        dt[k] = add2(dt[k], bias[k]);
        if (A.softplus) dt[k] = softplus(dt[k], slope ? slope + k : nullptr);
        else if (slope) slope[k] = f2(1.f);
    }
}
__device__ __forceinline__ float total(F2 a) {
    float x, y;
    parts(a, x, y);
    return x + y;
}

// v0 and v1 summed over two lanes that differ in `bit`: the lane without it keeps v0's sum.
__device__ __forceinline__ float halve(float v0, float v1, int lane, int bit) {
    const bool up = lane & bit;
    const float keep = up ? v1 : v0, give = up ? v0 : v1;
    return keep + __shfl_xor_sync(ALL, give, bit);
}

// Where a CTA works: a tile of CT channels of one group, one sequence, one segment of the time axis. Its threads have two
// tasks: the states of one channel on L lanes each, and V channels of the tile's tokens each, PI of them. W warps: 8, or 2 where a group
// has few channels.
template <int L, int W>
struct Place {
    static constexpr int NT = 32 * W, CH = 32 / L, CT = W * CH, V = sel_width(L), P = (V + 1) / 2;
    static constexpr int QUADS = CT / V, ROWS = NT / QUADS, PI = (TT + ROWS - 1) / ROWS;
    static constexpr int CTP = CT + CH;              // floats from lane to lane of the sums over n: lanes apart in the banks
    static constexpr int DW = CT + (V > 1 ? 4 * V : 0);  // a token's entries of du
    int b, s, ct, g, c0, cend, t0, t1, te;           // tokens t0..t1, te: up to the sequence's end
    int lane, gl, cl, c, ch, first, row;             // states' lane, channel; the V channels' first in the tile, and first row
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
        first = threadIdx.x % QUADS * V, row = threadIdx.x / QUADS;
    }
    __device__ __forceinline__ int column() const { return c0 + first; }
    __device__ __forceinline__ int width() const { return min(V, max(0, cend - column())); }  // of the V channels, inside the group
    // where channel c of a token stands in du: the V of a thread apart, so that neither writes nor reads meet in a bank
    static constexpr int STEP = QUADS + (V > 1 ? 4 : 0);
    static __device__ __forceinline__ int entry(int c) { return c % V * STEP + c / V; }
    // the thread's entries: (d, u) of every channel
    __device__ __forceinline__ void write(float2* du, int r, const F2* d, const F2* u) const {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float d0, d1, u0, u1;
            parts(d[k / 2], d0, d1), parts(u[k / 2], u0, u1);
            du[r * DW + k * STEP + first / V] = make_float2(k & 1 ? d1 : d0, k & 1 ? u1 : u0);
        }
    }
};
// V floats of the thread's own channels in shared memory, [token][CT]
template <int V>
__device__ __forceinline__ void own_write(float* p, const F2* f) {
    if constexpr (V == 4) *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(f[0].v, f[1].v);
    else if constexpr (V == 2) *reinterpret_cast<unsigned long long*>(p) = f[0].v;
    else {
        float a, b;
        parts(f[0], a, b);
        *p = a;
    }
}
template <int V>
__device__ __forceinline__ void own_read(const float* p, F2* f) {
    if constexpr (V == 4) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p);
        f[0].v = t.x, f[1].v = t.y;
    } else if constexpr (V == 2) {
        f[0].v = *reinterpret_cast<const unsigned long long*>(p);
    } else {
        f[0] = f2(*p, 0.f);
    }
}
// The sums over a channel's L lanes: [L][CTP] of a token, the thread's V channels
template <int L, int W>
__device__ __forceinline__ void lane_sums(const float* p, F2* f) {
    using P = Place<L, W>;
    own_read<P::V>(p, f);
#pragma unroll
    for (int l = 1; l < L; ++l) {
        F2 t[P::P];
        own_read<P::V>(p + l * P::CTP, t);
#pragma unroll
        for (int k = 0; k < P::P; ++k) f[k] = add2(f[k], t[k]);
    }
}
template <int V>
__device__ __forceinline__ void load_columns(const float* p, int at, int n, F2* f) {
    const Raw<float, V> r = load<false, float, V>(p + at, p ? n : 0);
    values<float, V>(r, f);
}

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
// M tokens' (dt, u) and b as they stand in shared memory, with the tokens' strides, and from them the decays and the writes u b.
// Read and worked on apart, so that the reads can go before the stores of the tokens before.
template <int M, int S>
struct Tokens {
    static constexpr int H = S / 2;
    float2 du[M];
    F2 u[M][H], a[M][H];
    __device__ __forceinline__ void read(const float2* d, int dstride, const float* v, int vstride) {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            du[j] = d[j * dstride];
            read_vec<S>(v + j * vstride, u[j]);
        }
    }
    __device__ __forceinline__ void work(const F2* A2) {
        F2 t[M * H];
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int k = 0; k < H; ++k) t[j * H + k] = mul2(f2(du[j].x), A2[k]), u[j][k] = mul2(f2(du[j].y), u[j][k]);
        decay<M * H>(t);
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int k = 0; k < H; ++k) a[j][k] = t[j * H + k];
    }
};
template <int M, int S>
__device__ __forceinline__ void decays(const float2* du, int dstride, const float* v, int vstride, const F2* A2, F2 (*a)[S / 2],
                                       F2 (*u)[S / 2]) {
    Tokens<M, S> t;
    t.read(du, dstride, v, vstride);
    t.work(A2);
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
        for (int k = 0; k < S / 2; ++k) a[j][k] = t.a[j][k], u[j][k] = t.u[j][k];
}
// Four states' values of b or c of one token. VEC: N is a multiple of four and they can be read at once
template <bool VEC, class XT>
__device__ __forceinline__ void load_row(const XT* p, int n0, int N, float* v) {
    F2 f[2];
    values<XT, 4>(load<VEC, XT, 4>(p + n0, N - n0), f);
    parts(f[0], v[0], v[1]), parts(f[1], v[2], v[3]);
}
// A tile's rows of b or c: NB elements of [TT][NP] per thread.
template <int NP, int W>
struct Rows {
    static constexpr int NT = 32 * W, NB = (TT * NP + NT - 1) / NT;
};
template <bool VEC, class XT, int NP, int W>
__device__ __forceinline__ void fetch_rows(const XT* p, long long ts, int tb, int te, int N, XT* r) {
    constexpr int NT = 32 * W;
#pragma unroll
    for (int k = 0; k < Rows<NP, W>::NB; ++k) {
        const int i = threadIdx.x + k * NT, t = i / NP, n = i % NP;
        r[k] = XT();
        if ((TT * NP % NT == 0 || t < TT) && tb + t < te && n < N) r[k] = *token<VEC>(p, n, tb + t, ts);
    }
}

// A segment's own state and what is left of the one that entered it. The decays of a segment together may be past the largest number where
// A or dt has the other sign; a state of 0 stays 0 all the same.
__device__ __forceinline__ float pass_on(float h, float keep, float own) { return h == 0.f ? own : fmaf(keep, h, own); }

// The state that enters the CTA's segment (REV: the cotangent that enters it from behind), of the thread's S states as they stand in
// memory: the sequence's own, then through the segments before it, each with its own state from 0 and the sum of its steps; or, where there are
// many segments or the final state overwrites h0, as join_kernel has left it.
template <int L, int W, int S, bool REV>
__device__ __forceinline__ void entering(const SelArgs& A, const Place<L, W>& p, int n0, const float* a2, float* h) {
    const long long EN = (long long)A.E * A.N, own = (long long)p.ch * A.N;
#pragma unroll
    for (int k = 0; k < S; ++k) h[k] = 0.f;
    if (!p.live) return;
    const float* first = REV ? A.dh_T : A.h0;
    if (A.joined) load_states<S>(A.seg_state + ((long long)p.b * A.nseg + p.s) * EN + own, n0, A.N, A.vec_n, h);
    else if (first) load_states<S>(first + p.b * EN + own, n0, A.N, A.vec_n, h);
    if (A.joined || A.nseg == 1) return;
    const int n = REV ? A.nseg - 1 - p.s : p.s;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const long long at = (long long)p.b * A.nseg + (REV ? A.nseg - 1 - i : i);
        const float sum = A.seg_sum[at * A.E + p.ch];
        float v[S];
        load_states<S>(A.seg_state + at * EN + own, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < S; ++k) h[k] = pass_on(h[k], ex2(a2[k] * sum), v[k]);
    }
}

// ---- forward: all tokens of a segment, from the state that enters it
// Between two barriers a CTA finishes the tile before, prepares the next one (in the other buffers) and works on its own.
template <class XT, int L, int S, int W>
struct FwdShared {
    static constexpr int NP = L * S, CT = Place<L, W>::CT;
    float2 du[2][TT * Place<L, W>::DW];             // (dt, u), u = dt x
    float gate[2][TT * CT], skip[2][TT * CT];    // silu(z) and skip x, for the thread that wrote them
    float b[2][TT * NP], c[2][TT * NP];
    float y[2][TT * L * Place<L, W>::CTP];          // the lanes' parts of the sums over n
};

template <class XT, int L, int S, int W, bool VEC>
__global__ void __launch_bounds__(32 * W, 16 / W) fwd_kernel(const SelArgs A) {
    using P = Place<L, W>;
    constexpr int NT = P::NT, NP = L * S, CT = P::CT, CTP = P::CTP, PI = P::PI, NB = Rows<NP, W>::NB, H = S / 2, V = P::V, Q = P::P;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    FwdShared<XT, L, S, W>& sh = *reinterpret_cast<FwdShared<XT, L, S, W>*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * S, pw = p.width();
    F2 h[H], A2[H], bias[Q], skip[Q];
    {
        float v[S] = {};
        if (p.live) load_states<S>(A.A + (long long)p.ch * A.N, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] *= kLog2e;
        pack<S>(v, A2);
        float e[S];
        entering<L, W, S, false>(A, p, n0, v, e);
        pack<S>(e, h);
        load_columns<V>(A.dt_bias, p.column(), pw, bias);
        load_columns<V>(A.skip, p.column(), pw, skip);
    }
    const XT *xp = static_cast<const XT*>(A.x) + p.b * A.xbs, *zp = static_cast<const XT*>(A.z) + p.b * A.zbs,
             *bp = static_cast<const XT*>(A.b) + p.b * A.bbs + (long long)p.g * A.N, *cp = static_cast<const XT*>(A.c) + p.b * A.cbs + (long long)p.g * A.N;
    const void* dp = dt_at<XT>(A, p.b);
    XT* yp = static_cast<XT*>(A.y) + (long long)p.b * A.T * A.E;
    Raw<XT, V> rx[PI], rz[PI];
    Raw<float, V> rd[PI];
    XT rb[NB], rc[NB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load<VEC, XT, V>(token<VEC>(xp, p.column(), t, A.xts), n);
            rd[k] = load_dt<VEC, XT, V>(A, dp, p.column(), t, n);
            if (A.z) rz[k] = load<VEC, XT, V>(token<VEC>(zp, p.column(), t, A.zts), n);
        }
        fetch_rows<VEC, XT, NP, W>(bp, A.bts, tb, p.te, A.N, rb);
        fetch_rows<VEC, XT, NP, W>(cp, A.cts, tb, p.te, A.N, rc);
    };
    auto prepare = [&](int tb, int buf) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (TT % P::ROWS != 0 && r >= TT) continue;
            F2 dt[Q], x[Q], u[Q];
            step_sizes<XT, V>(A, rd[k], bias, dt, nullptr);
            values<XT, V>(rx[k], x);
            const bool in = tb + r < p.te;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!in) dt[q] = f2(0.f);
                u[q] = mul2(dt[q], x[q]);  // rows behind the end were read as 0
            }
            p.write(sh.du[buf], r, dt, u);
            if (!A.y) continue;
            if (A.skip) {
#pragma unroll
                for (int q = 0; q < Q; ++q) x[q] = mul2(x[q], skip[q]);
                own_write<V>(sh.skip[buf] + r * CT + p.first, x);
            }
            if (A.z) {
                values<XT, V>(rz[k], x);
#pragma unroll
                for (int q = 0; q < Q; ++q) x[q] = mul2(x[q], sigmoid(x[q]));
                own_write<V>(sh.gate[buf] + r * CT + p.first, x);
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i < TT * NP) sh.b[buf][i] = to_f(rb[k]), sh.c[buf][i] = to_f(rc[k]);
        }
    };
    auto finish = [&](int tb, int buf) {  // the tile's outputs
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r;
            if (r >= TT || t >= p.te) continue;
            F2 y[Q], f[Q];
            lane_sums<L, W>(sh.y[buf] + r * L * CTP + p.first, y);
            if (A.skip) {
                own_read<V>(sh.skip[buf] + r * CT + p.first, f);
#pragma unroll
                for (int q = 0; q < Q; ++q) y[q] = add2(y[q], f[q]);
            }
            if (A.z) {
                own_read<V>(sh.gate[buf] + r * CT + p.first, f);
#pragma unroll
                for (int q = 0; q < Q; ++q) y[q] = mul2(y[q], f[q]);
            }
            store<VEC, XT, V>(token<VEC>(yp, p.column(), t, A.E), y, pw);
        }
    };
    const int tiles = (p.te - p.t0 + TT - 1) / TT, entry = P::entry(p.c);
    float* mark = A.marks + (((long long)p.b * A.nmarks + p.t0 / kSelMark) * A.E + p.ch) * A.N;
    const bool marks = A.marks && p.live;
    if (tiles > 0) fetch(p.t0), prepare(p.t0, 0);
    if (tiles > 1) fetch(p.t0 + TT);
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int tb = p.t0 + i * TT, buf = i & 1;
        if (i > 0 && A.y) finish(tb - TT, buf ^ 1);
        if (i + 1 < tiles) prepare(tb + TT, buf ^ 1);
        if (i + 2 < tiles) fetch(tb + 2 * TT);
        float* ys = sh.y[buf] + p.gl * CTP + p.c;
        const float2* du = sh.du[buf] + entry;
        const float *vb = sh.b[buf] + n0, *vc = sh.c[buf] + n0;
        F2 kept[TT / kSelMark][H];
        Tokens<4, S> now, next;
        now.read(du, P::DW, vb, NP);
        now.work(A2);
#pragma unroll
        for (int q = 0; q < TT; q += 4) {
            F2 cv[4][H];
            if (q + 4 < TT) next.read(du + (q + 4) * P::DW, P::DW, vb + (q + 4) * NP, NP);
#pragma unroll
            for (int j = 0; j < 4; ++j) read_vec<S>(vc + (q + j) * NP, cv[j]);
            if (q + 4 < TT) next.work(A2);  // beside the chain below
            if (q % kSelMark == 0)
#pragma unroll
                for (int k = 0; k < H; ++k) kept[q / kSelMark][k] = h[k];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                F2 yy;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    h[k] = fma2(now.a[j][k], h[k], now.u[j][k]);
                    yy = k ? fma2(h[k], cv[j][k], yy) : mul2(h[k], cv[j][k]);
                }
                ys[(q + j) * L * CTP] = total(yy);
            }
            now = next;
        }
        if (marks) {
#pragma unroll
            for (int m = 0; m < TT / kSelMark; ++m, mark += (long long)A.E * A.N) {
                float v[S];
                unpack<S>(kept[m], v);
                if (tb + m * kSelMark < p.te) store_states<S>(mark, n0, A.N, A.vec_n, v);
            }
        }
        __syncthreads();
    }
    if (A.y) {
        if (tiles > 0) finish(p.t0 + (tiles - 1) * TT, (tiles - 1) & 1);
        const F2 zero[Q] = {};
        for (int t = p.te + p.row; t < p.t1; t += P::ROWS)  // behind the sequence's end
            store<VEC, XT, V>(token<VEC>(yp, p.column(), t, A.E), zero, pw);
    }
    if (A.h_out && p.s == A.nseg - 1 && p.live) {
        float v[S];
        unpack<S>(h, v);
        store_states<S>(A.h_out + ((long long)p.b * A.E + p.ch) * A.N, n0, A.N, A.vec_n, v);
    }
}

// ---- a segment's state from 0 at its end (REV: the cotangent from 0 at its start) and the sum of its dt
template <class XT, int L, int S, int W>
struct SegShared {
    static constexpr int NP = L * S;
    float2 du[2][TT * Place<L, W>::DW];       // (dt, w), w = dt x or dy silu(z)
    float v[2][TT * NP];                   // b or c
    float sum[32 * W * 4];
};

template <class XT, int L, int S, int W, bool REV, bool VEC>
__global__ void __launch_bounds__(32 * W, 16 / W) seg_kernel(const SelArgs A) {
    using P = Place<L, W>;
    constexpr int NT = P::NT, NP = L * S, PI = P::PI, NB = Rows<NP, W>::NB, H = S / 2, V = P::V, Q = P::P;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    SegShared<XT, L, S, W>& sh = *reinterpret_cast<SegShared<XT, L, S, W>*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * S, pw = p.width();
    F2 h[H], A2[H], bias[Q], sum[Q];
    {
        float v[S] = {};
        if (p.live) load_states<S>(A.A + (long long)p.ch * A.N, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] *= kLog2e;
        pack<S>(v, A2);
#pragma unroll
        for (int k = 0; k < H; ++k) h[k] = f2(0.f);
        load_columns<V>(A.dt_bias, p.column(), pw, bias);
#pragma unroll
        for (int q = 0; q < Q; ++q) sum[q] = f2(0.f);
    }
    const XT *xp = static_cast<const XT*>(REV ? A.dy : A.x) + p.b * (REV ? A.ybs : A.xbs),
             *zp = static_cast<const XT*>(A.z) + p.b * A.zbs,
             *vp = static_cast<const XT*>(REV ? A.c : A.b) + p.b * (REV ? A.cbs : A.bbs) + (long long)p.g * A.N;
    const void* dp = dt_at<XT>(A, p.b);
    const long long xts = REV ? A.yts : A.xts, vts = REV ? A.cts : A.bts;
    const bool gated = REV && A.z;
    Raw<XT, V> rx[PI], rz[PI];
    Raw<float, V> rd[PI];
    XT rv[NB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load<VEC, XT, V>(token<VEC>(xp, p.column(), t, xts), n);
            rd[k] = load_dt<VEC, XT, V>(A, dp, p.column(), t, n);
            if (gated) rz[k] = load<VEC, XT, V>(token<VEC>(zp, p.column(), t, A.zts), n);
        }
        fetch_rows<VEC, XT, NP, W>(vp, vts, tb, p.te, A.N, rv);
    };
    auto prepare = [&](int tb, int buf) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (TT % P::ROWS != 0 && r >= TT) continue;
            F2 dt[Q], w[Q], z[Q];
            step_sizes<XT, V>(A, rd[k], bias, dt, nullptr);
            values<XT, V>(rx[k], w);
            if (gated) values<XT, V>(rz[k], z);
            const bool in = tb + r < p.te;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!in) dt[q] = f2(0.f);
                if constexpr (!REV) w[q] = mul2(w[q], dt[q]);
                else if (gated) w[q] = mul2(w[q], mul2(z[q], sigmoid(z[q])));
                sum[q] = add2(sum[q], dt[q]);
            }
            p.write(sh.du[buf], r, dt, w);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i < TT * NP) sh.v[buf][i] = to_f(rv[k]);
        }
    };
    const int tiles = (p.te - p.t0 + TT - 1) / TT, entry = P::entry(p.c);
    auto base = [&](int i) { return p.t0 + (REV ? tiles - 1 - i : i) * TT; };
    if (tiles > 0) fetch(base(0)), prepare(base(0), 0);
    if (tiles > 1) fetch(base(1));
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int buf = i & 1;
        if (i + 1 < tiles) prepare(base(i + 1), buf ^ 1);
        if (i + 2 < tiles) fetch(base(i + 2));
        const float2* du = sh.du[buf] + entry;
        const float* v = sh.v[buf] + n0;
        Tokens<4, S> now, next;
        now.read(du + (REV ? TT - 4 : 0) * P::DW, P::DW, v + (REV ? TT - 4 : 0) * NP, NP);
        now.work(A2);
#pragma unroll
        for (int i4 = 0; i4 < TT; i4 += 4) {
            const int q = REV ? TT - 8 - i4 : i4 + 4;
            if (i4 + 4 < TT) {
                next.read(du + q * P::DW, P::DW, v + q * NP, NP);
                next.work(A2);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    if constexpr (REV) h[k] = mul2(now.a[3 - j][k], add2(now.u[3 - j][k], h[k]));
                    else h[k] = fma2(now.a[j][k], h[k], now.u[j][k]);
                }
            now = next;
        }
        __syncthreads();
    }
    const long long at = (long long)(p.b * A.nseg + p.s) * A.E;
    if (p.live) {
        float v[S];
        unpack<S>(h, v);
        store_states<S>(A.seg_state + (at + p.ch) * A.N, n0, A.N, A.vec_n, v);
    }
    own_write<V>(sh.sum + threadIdx.x * V, sum);
    __syncthreads();
    if (p.row == 0) {  // row by row, in order
        for (int r = 1; r < P::ROWS; ++r) {
            F2 o[Q];
            own_read<V>(sh.sum + (r * P::QUADS + threadIdx.x) * V, o);
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[q] = add2(sum[q], o[q]);
        }
        store<false, float, V>(A.seg_sum + at + p.column(), sum, pw);
    }
}

// The states that enter the segments (REV: the cotangents that enter them from behind), in place: for more than kSelFold segments, which
// take longer to go through than a launch, and for a final state that overwrites h0, which CTAs still to come could not read any more.
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
        const float own = *p, keep = ex2(a * A.seg_sum[at * A.E + e]);
        *p = h;
        h = pass_on(h, keep, own);
    }
}

// ---- one token: 4 states per thread, L lanes per channel, R sequences. What belongs to a channel is computed by one of its
// lanes for each sequence: dt, x, the gate and the output of sequence k by lane k % L (of the first four). With R = 4 the lanes' sums
// over n end with those lanes, and a state costs a fourth of the instructions around it.
template <class XT, int L, int R, bool VEC>
__global__ void __launch_bounds__(256) step_kernel(const SelArgs A) {
    constexpr int LR = L < R ? L : R, PR = R / LR;  // lanes with sequences of their own, and how many of these
    const unsigned per = (unsigned)(((long long)A.E * L + 255) / 256), blk = blockIdx.x / per;  // CTAs per R sequences
    const long long i = (long long)(blockIdx.x - blk * per) * 256 + threadIdx.x;
    const int gl = (int)(threadIdx.x % L), n0 = gl * 4, lane = threadIdx.x & 31;
    const bool in = i / L < A.E;
    const int e = in ? (int)(i / L) : 0, g = A.G == 1 ? 0 : e / A.Eg;
    const int b0 = (int)blk * R, most = A.B - 1;  // sequences past the last read the last one's
    const int live = !in ? 0 : min(R, A.B - b0);
    const long long EN = (long long)A.E * A.N, own = (long long)e * A.N;
    float a[4], dt[PR], u[PR], x[PR], z[PR], h[R][4], bv[R][4], cv[R][4];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const long long b = min(b0 + k, most);
        load_states<4>(A.h0 + b * EN + own, n0, A.N, VEC, h[k]);
        load_row<VEC>(static_cast<const XT*>(A.b) + b * A.bbs + (long long)g * A.N, n0, A.N, bv[k]);
        load_row<VEC>(static_cast<const XT*>(A.c) + b * A.cbs + (long long)g * A.N, n0, A.N, cv[k]);
    }
    load_states<4>(A.A + own, n0, A.N, VEC, a);
    const float bias = A.dt_bias ? A.dt_bias[e] : 0.f, skip = A.skip ? A.skip[e] : 0.f;
#pragma unroll
    for (int j = 0; j < PR; ++j) {
        const long long b = min(b0 + gl % LR + j * LR, most);
        x[j] = to_f(static_cast<const XT*>(A.x)[b * A.xbs + e]);
        z[j] = A.z ? to_f(static_cast<const XT*>(A.z)[b * A.zbs + e]) : 0.f;
        const long long di = b * A.dbs + e;
        dt[j] = sizeof(XT) == 4 || A.dt32 ? static_cast<const float*>(A.dt)[di] : to_f(static_cast<const XT*>(A.dt)[di]);
    }
#pragma unroll
    for (int j = 0; j < PR; ++j) {
        dt[j] += bias;
        if (A.softplus) {
            float other;
            parts(softplus(f2(dt[j], 0.f), nullptr), dt[j], other);
        }
        u[j] = dt[j] * x[j];
    }
    const F2 a01 = f2(a[0] * kLog2e, a[1] * kLog2e), a23 = f2(a[2] * kLog2e, a[3] * kLog2e);
    float y[R];
    float* to = A.h_out + b0 * EN + own;
#pragma unroll
    for (int k = 0; k < R; ++k, to += EN) {
        float d = dt[k / LR], v = u[k / LR];
        if constexpr (LR > 1) {
            d = __shfl_sync(ALL, d, (lane & ~(L - 1)) + k % LR);
            v = __shfl_sync(ALL, v, (lane & ~(L - 1)) + k % LR);
        }
        F2 t[2] = {mul2(f2(d), a01), mul2(f2(d), a23)};
        decay<2>(t);
        const F2 h01 = fma2(t[0], f2(h[k][0], h[k][1]), mul2(f2(v), f2(bv[k][0], bv[k][1])));
        const F2 h23 = fma2(t[1], f2(h[k][2], h[k][3]), mul2(f2(v), f2(bv[k][2], bv[k][3])));
        y[k] = total(fma2(h23, f2(cv[k][2], cv[k][3]), mul2(h01, f2(cv[k][0], cv[k][1]))));
        parts(h01, h[k][0], h[k][1]), parts(h23, h[k][2], h[k][3]);
        if (k < live) store_states<4>(to, n0, A.N, VEC, h[k]);
    }
    // the lanes' sums, each to the lane of its sequence
    if constexpr (R == 4 && L > 1) {
        y[0] = halve(y[0], y[1], lane, 1), y[2] = halve(y[2], y[3], lane, 1);
        if constexpr (L == 2) {
            y[1] = y[2];
        } else {
            y[0] = halve(y[0], y[2], lane, 2);
#pragma unroll
            for (int o = 4; o < L; o *= 2) y[0] += __shfl_xor_sync(ALL, y[0], o);
        }
    } else if constexpr (R == 1) {
#pragma unroll
        for (int o = 1; o < L; o *= 2) y[0] += __shfl_xor_sync(ALL, y[0], o);
    }
    if (gl >= LR) return;
#pragma unroll
    for (int j = 0; j < PR; ++j) {
        const int k = gl + j * LR;
        if (k >= live) continue;
        if (A.skip) y[j] = fmaf(skip, x[j], y[j]);
        if (A.z) y[j] *= z[j] * rcp(1.f + ex2(-z[j] * kLog2e));
        put(static_cast<XT*>(A.y) + (long long)(b0 + k) * A.E + e, y[j]);
    }
}

}  // namespace selective
}  // namespace lattice

// short_conv.cuh -- short causal convolution of every channel over the tokens of a sequence, its
// backward pass and its single-token step (sm_100a).
//
//   v_t = bias + sum_k w[k] x_{t-K+1+k},  y_t = act(v_t);  x before the first token: the state, or 0
// Backward, with e_t = dy_t act'(v_t):
//   dx_s = sum_j w[K-1-j] e_{s+j},  dw[k] = sum_t e_t x_{t-K+1+k},  dbias = sum_t e_t
//
// HBM bounds it: x is read once and y written once. A thread has V neighbouring channels and
// walks down a run of tokens with the last K-1 inputs in registers, loads of the next U tokens under way
// at once; a run's K-1 first inputs are its neighbour's last ones and mostly come from the L2. The mid-size layer (8 x 4096 tokens of
// 2048 bf16 channels, 4 taps) takes 53.5 us forward, 5.0 TB/s of what has to move, with the special function units 59 % busy (the SiLU's
// exponential and reciprocal); backward 108 us, 3.7 TB/s, where a token's 117 instructions bind at 16 warps per SM (a thread's 128 registers
// hold weights, window, slopes and sums; copies through shared memory keep loads out of them). One token of 256 sequences of
// 4096 channels takes 5 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "args.h"
#include "f32x2.cuh"

namespace lattice {
namespace conv {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float& p, float v) { p = v; }
__device__ __forceinline__ void put(__nv_bfloat16& p, float v) { p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half& p, float v) { p = __float2half_rn(v); }

// A thread's V channels in H numbers: one, or pairs in packed instructions
template <int V>
struct Numbers {
    using N = F2;
    static constexpr int H = V / 2;
};
template <>
struct Numbers<1> {
    using N = float;
    static constexpr int H = 1;
};
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 mad(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ F2 mul(F2 a, F2 b) { return mul2(a, b); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ F2 add(F2 a, F2 b) { return add2(a, b); }
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-1.442695041f * v)); }
__device__ __forceinline__ F2 sigmoid(F2 v) { return each(each(mul2(v, f2(-1.442695041f)), [](float n) { return 1.f + ex2(n); }), rcp); }
__device__ __forceinline__ void fill(float& n, float v) { n = v; }
__device__ __forceinline__ void fill(F2& n, float v) { n = f2(v); }

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};
template <class T, int V>
__device__ __forceinline__ Vec<T, V> load(const void* p, long long i) {
    return *reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(p) + i);
}
template <class T, int V>
__device__ __forceinline__ void store(void* p, long long i, const typename Numbers<V>::N* n) {
    Vec<T, V> r;
    if constexpr (V == 1) {
        put(r.v[0], n[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            float a, b;
            parts(n[k], a, b);
            if constexpr (std::is_same<T, __half>::value) *reinterpret_cast<__half2*>(&r.v[2 * k]) = __floats2half2_rn(a, b);
            else if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(&r.v[2 * k]) = __floats2bfloat162_rn(a, b);
            else r.v[2 * k] = a, r.v[2 * k + 1] = b;
        }
    }
    *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(p) + i) = r;
}
template <class T, int V>
__device__ __forceinline__ void values(const Vec<T, V>& r, typename Numbers<V>::N* n) {
    if constexpr (V == 1) {
        n[0] = to_f(r.v[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) n[k] = f2(to_f(r.v[2 * k]), to_f(r.v[2 * k + 1]));
    }
}
template <class T, int V>
__device__ __forceinline__ Vec<T, V> zeros() {
    Vec<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) put(r.v[v], 0.f);
    return r;
}
// N consecutive weights, N a multiple of V, as vectors of V
template <class T, int V, int N>
__device__ __forceinline__ void weight_run(const void* p, long long i, float* f) {
#pragma unroll
    for (int k = 0; k < N; k += V) {
        const Vec<T, V> r = load<T, V>(p, i + k);
#pragma unroll
        for (int v = 0; v < V; ++v) f[k + v] = to_f(r.v[v]);
    }
}
// A thread's weights, from the oldest input's on, and bias
template <class XT, int K, int V>
__device__ __forceinline__ void weights(const ConvArgs& A, int c, typename Numbers<V>::N (*w)[Numbers<V>::H], typename Numbers<V>::N* bias) {
    float f[K * V], g[V] = {};
    if (sizeof(XT) == 4 || A.w32) {
        weight_run<float, V, K * V>(A.w, (long long)c * K, f);
        if (A.bias) weight_run<float, V, V>(A.bias, c, g);
    } else {
        weight_run<XT, V, K * V>(A.w, (long long)c * K, f);
        if (A.bias) weight_run<XT, V, V>(A.bias, c, g);
    }
    if constexpr (V == 1) {
        bias[0] = g[0];
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][0] = f[k];
    } else {
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
            bias[h] = f2(g[2 * h], g[2 * h + 1]);
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][h] = f2(f[2 * h * K + k], f[(2 * h + 1) * K + k]);
        }
    }
}

// The thread's next D tokens of one array on their way through shared memory, in groups of U: cp.async needs no registers, and
// since every thread reads what it copied itself, no barrier. Pieces of less than 4 bytes (one 16-bit channel per
// thread) cannot be copied so; they are loaded U tokens ahead of the work.
template <class T, int V, int U, int D>
struct Ahead {
    static constexpr bool RING = sizeof(T) * V >= 4;
    static constexpr int BYTES = RING ? D * 256 * (int)sizeof(T) * V : 16;
    uint32_t slot;
    Vec<T, V> next[RING ? 1 : U];
    __device__ __forceinline__ explicit Ahead(const Vec<T, V>* ring) {
        slot = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
    }
    // group g's U tokens, of which `n` are there, the first at p
    __device__ __forceinline__ void fetch(int g, const T* p, long long ts, int n) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (j >= n) continue;
            if constexpr (RING) {
                const uint32_t to = slot + ((g * U + j) % D) * 256 * (uint32_t)sizeof(Vec<T, V>);
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p + j * ts), "n"((int)sizeof(Vec<T, V>)) : "memory");
            } else {
                next[j] = load<T, V>(p, j * ts);
            }
        }
    }
    __device__ __forceinline__ void take(int g, const Vec<T, V>* ring, Vec<T, V>* r) const {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if constexpr (RING) r[j] = ring[((g * U + j) % D) * 256 + threadIdx.x];
            else r[j] = next[j];
        }
    }
};
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Who does what: V channels and a run of A.run tokens of one sequence per thread.
template <int V>
struct Place {
    int c, run, b, len;
    bool in;
    __device__ __forceinline__ Place(const ConvArgs& A) {
        const unsigned cv = A.C / V;
        const unsigned long long i = (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x, r = i / cv;
        c = (int)(i - r * cv) * V;
        in = r < (unsigned long long)A.B * A.runs;
        b = (int)(r / A.runs), run = (int)(r - (unsigned long long)b * A.runs);
        len = A.lengths && in ? min(max(A.lengths[b], 0), A.T) : A.T;
    }
};
// Input row t (t >= -(K-1)): before the first token the state's, or 0
template <class XT, int K, int V>
__device__ __forceinline__ Vec<XT, V> input(const ConvArgs& A, int b, int c, int t) {
    if (t >= 0) return load<XT, V>(A.x, b * A.xbs + t * A.xts + c);
    return A.state ? load<XT, V>(A.state, ((long long)b * (K - 1) + K - 1 + t) * A.C + c) : zeros<XT, V>();
}

template <class XT, int K, int V>
__global__ void __launch_bounds__(256, conv_resident(false, K)) fwd_kernel(const ConvArgs A) {
    using N = typename Numbers<V>::N;
    // Tokens whose loads are under way at once: two of 16 bytes do beside the lines brought nearer, with fewer spills (8 x 4096 tokens of 1024
    // fp32 channels, 3 taps: 51.5 -> 48.6 us); without those lines four (5 to 8 taps: 50, 50, 50 and 53 us, with two 60, 60, 61 and 63 us).
    constexpr int U = sizeof(XT) * V > 8 && K <= 4 ? 2 : 4, H = Numbers<V>::H;
    const Place<V> p(A);
    if (!p.in) return;
    N w[K][H], bias[H], win[K][H];  // win[k]: x_{t-K+1+k}
    weights<XT, K, V>(A, p.c, w, bias);
    const int t0 = p.run * A.run, t1 = min(A.T, t0 + A.run), te = min(t1, p.len);
    const bool tail = p.run == 0 && A.state_out;  // writes the state at the sequence's end
    Vec<XT, V> last[K > 1 ? K - 1 : 1];
    if (tail && p.len < K - 1) {  // part of the state itself: read before anything is written, which may be in place
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j] = input<XT, K, V>(A, p.b, p.c, p.len - (K - 1) + j);
    }
    if (t0 < te) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) values<XT, V>(input<XT, K, V>(A, p.b, p.c, t0 - (K - 1) + k), win[k]);
    }
    const XT* x = static_cast<const XT*>(A.x) + p.b * A.xbs + p.c + (long long)t0 * A.xts;
    XT* y = static_cast<XT*>(A.y) + ((long long)p.b * A.T + t0) * A.C + p.c;
    auto token = [&](const Vec<XT, V>& r) {
        N s[H];
        values<XT, V>(r, win[K - 1]);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            s[h] = bias[h];
#pragma unroll
            for (int k = 0; k < K; ++k) s[h] = mad(w[k][h], win[k][h], s[h]);
            if (A.silu) s[h] = mul(s[h], sigmoid(s[h]));
#pragma unroll
            for (int k = 0; k < K - 1; ++k) win[k][h] = win[k + 1][h];
        }
        store<XT, V>(y, 0, s);
        y += A.C;
    };
    int t = t0;
    Vec<XT, V> r[U], next[U];  // U tokens' loads are under way while U tokens are worked on
    auto fetch = [&](Vec<XT, V>* to) {
#pragma unroll
        for (int j = 0; j < U; ++j) to[j] = load<XT, V>(x, j * A.xts);
        x += U * A.xts;
    };
    // The U tokens after those are brought into the L2, which takes no registers (mid-size layer 55.9 -> 53.5 us; 2051 channels,
    // call included, 113 -> 102 us). With more taps a token's arithmetic hides the way, and they cost more than
    // they give (8 x 4096 tokens, 5 to 8 taps: 2048 bf16 channels 62.5, 63.5, 65 and 69.5 us, with them 64.5, 67.5, 71 and 77 us; 1024 fp32
    // channels 50 to 53 us, with them 50 to 55 us), but for single 16-bit elements (2051 channels: 92, 92, 123 and 124 us, with them 85, 95, 104
    // and 102 us), which are not told apart.
    auto ahead = [&]() {
#pragma unroll
        for (int j = 0; j < U; ++j) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + j * A.xts));
    };
    if (t + U <= te) fetch(r);
#pragma unroll 1
    for (; t + U <= te; t += U) {
        if (t + 2 * U <= te) fetch(next);
        if (K <= 4 && t + 3 * U <= te) ahead();
#pragma unroll
        for (int j = 0; j < U; ++j) token(r[j]), r[j] = next[j];
    }
#pragma unroll 1
    for (; t < te; ++t, x += A.xts) token(load<XT, V>(x, 0));
    N zero[H];
#pragma unroll
    for (int h = 0; h < H; ++h) fill(zero[h], 0.f);
#pragma unroll 1
    for (t = max(t0, te); t < t1; ++t, y += A.C) store<XT, V>(y, 0, zero);  // behind the end
    if (!tail) return;
    if (p.len >= K - 1) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j] = load<XT, V>(A.x, p.b * A.xbs + (long long)(p.len - (K - 1) + j) * A.xts + p.c);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        *reinterpret_cast<Vec<XT, V>*>(static_cast<XT*>(A.state_out) + ((long long)p.b * (K - 1) + j) * A.C + p.c) = last[j];
}

// One token: the state's rows move up by one
template <class XT, int K, int V>
__global__ void __launch_bounds__(256) step_kernel(const ConvArgs A) {
    using N = typename Numbers<V>::N;
    constexpr int H = Numbers<V>::H;
    const Place<V> p(A);
    if (!p.in) return;
    N w[K][H], y[H], x[H];
    Vec<XT, V> r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) r[k] = input<XT, K, V>(A, p.b, p.c, k - (K - 1));
    weights<XT, K, V>(A, p.c, w, y);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        values<XT, V>(r[k], x);
#pragma unroll
        for (int h = 0; h < H; ++h) y[h] = mad(w[k][h], x[h], y[h]);
    }
    if (A.silu)
#pragma unroll
        for (int h = 0; h < H; ++h) y[h] = mul(y[h], sigmoid(y[h]));
    store<XT, V>(A.y, (long long)p.b * A.C + p.c, y);
#pragma unroll
    for (int k = 1; k < K; ++k)
        *reinterpret_cast<Vec<XT, V>*>(static_cast<XT*>(A.state_out) + ((long long)p.b * (K - 1) + k - 1) * A.C + p.c) = r[k];
}

// A run's dx needs e of the K-1 tokens behind it, whose own inputs reach K-1 tokens back: x and dy of 2 (K-1)
// and K-1 tokens are read twice. The weights' gradients are summed over the run and written as
// one row [K+1][C] of the workspace per run.
template <class XT, int K, int V>
__global__ void __launch_bounds__(256, conv_resident(true, K)) bwd_kernel(const ConvArgs A) {
    using N = typename Numbers<V>::N;
    constexpr int U = 2, H = Numbers<V>::H, D = sizeof(XT) * V > 8 ? 4 : 8;
    using Q = Ahead<XT, V, U, D>;
    __shared__ __align__(16) Vec<XT, V> ring[Q::RING ? 2 * D * 256 : 1];
    const Place<V> p(A);
    if (!p.in) return;
    N w[K][H], bias[H], win[K][H], e[K][H], dw[K][H], db[H], one, minus;  // e[j]: e_{t-K+1+j}
    fill(one, 1.f), fill(minus, -1.f);
    weights<XT, K, V>(A, p.c, w, bias);
#pragma unroll
    for (int h = 0; h < H; ++h) {
        fill(db[h], 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) fill(e[k][h], 0.f), fill(dw[k][h], 0.f);
    }
    const int t0 = p.run * A.run, t1 = min(A.T, t0 + A.run), te = min(t1, p.len);
    const bool head = p.run == 0 && A.dstate;  // writes the gradients of the rows before the first token
    if (t0 < te) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) values<XT, V>(input<XT, K, V>(A, p.b, p.c, t0 - (K - 1) + k), win[k]);
    }
    const XT* x = static_cast<const XT*>(A.x) + p.b * A.xbs + p.c + (long long)t0 * A.xts;
    const XT* dy = static_cast<const XT*>(A.dy) + p.b * A.ybs + p.c + (long long)t0 * A.yts;
    XT* dx = static_cast<XT*>(A.dx) + ((long long)p.b * A.T + t0) * A.C + p.c;
    // e of the next token, from its x and dy; SUM: it is one of the run's
    auto forward = [&](const Vec<XT, V>& rx, const Vec<XT, V>& ry, bool sum) {
        values<XT, V>(rx, win[K - 1]);
        values<XT, V>(ry, e[K - 1]);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (A.silu) {
                N s = bias[h];
#pragma unroll
                for (int k = 0; k < K; ++k) s = mad(w[k][h], win[k][h], s);
                const N q = sigmoid(s);
                e[K - 1][h] = mul(e[K - 1][h], mad(mul(s, q), mad(q, minus, one), q));
            }
            if (sum) {
                db[h] = add(db[h], e[K - 1][h]);
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k][h] = mad(e[K - 1][h], win[k][h], dw[k][h]);
            }
        }
    };
    // the gradient of the token K - 1 back
    auto gradient = [&](N* d) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            d[h] = mul(w[K - 1][h], e[0][h]);
#pragma unroll
            for (int k = 1; k < K; ++k) d[h] = mad(w[K - 1 - k][h], e[k][h], d[h]);
        }
    };
    auto shift = [&]() {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int h = 0; h < H; ++h) win[k][h] = win[k + 1][h], e[k][h] = e[k + 1][h];
    };
    // the token t = s + K - 1, one at a time, and what the ends of run and sequence need
    auto careful = [&](int t) {
        if (t < p.len) {
            forward(load<XT, V>(x, 0), load<XT, V>(dy, 0), t < te);
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) fill(e[K - 1][h], 0.f);
        }
        x += A.xts, dy += A.yts;
        const int s = t - (K - 1);
        if (s >= t0 || head) {
            N d[H], more[H];
            gradient(d);
            const int j = s - (p.len - (K - 1));  // the final state's row
            if (A.dstate_out && j >= 0 && s < p.len) {
                values<XT, V>(load<XT, V>(A.dstate_out, ((long long)p.b * (K - 1) + j) * A.C + p.c), more);
#pragma unroll
                for (int h = 0; h < H; ++h) d[h] = add(d[h], more[h]);
            }
            if (s >= t0) store<XT, V>(dx, 0, d), dx += A.C;
            else store<XT, V>(A.dstate, ((long long)p.b * (K - 1) + K - 1 + s) * A.C + p.c, d);
        }
        shift();
    };
    const int end = t0 < te || head ? te + K - 1 : t0;
    int t = t0;
#pragma unroll 1
    for (; t < min(end, t0 + K - 1); ++t) careful(t);
    // tokens of the run whose K - 1 back are its own too, and no rows of the final state
    const int whole = A.dstate_out ? min(te, p.len - (K - 1)) : te;
    const int n = whole - t;
    if (n >= U) {
        Q qx(ring), qy(ring + (Q::RING ? D * 256 : 0));
        constexpr int G = Q::RING ? D / U - 1 : 1;  // groups ahead
        const int groups = n / U;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int m = g < groups ? U : 0;
            qx.fetch(g, x + g * U * A.xts, A.xts, m), qy.fetch(g, dy + g * U * A.yts, A.yts, m), commit();
        }
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            Vec<XT, V> rx[U], ry[U];
            const int m = g + G < groups ? U : 0;
            if constexpr (!Q::RING) qx.take(g, ring, rx), qy.take(g, ring, ry);
            qx.fetch(g + G, x + G * U * A.xts, A.xts, m), qy.fetch(g + G, dy + G * U * A.yts, A.yts, m), commit();
            if constexpr (Q::RING) {
                wait<G>();
                qx.take(g, ring, rx), qy.take(g, ring + D * 256, ry);
            }
            x += U * A.xts, dy += U * A.yts;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                N d[H];
                forward(rx[j], ry[j], true);
                gradient(d);
                store<XT, V>(dx, 0, d);
                dx += A.C;
                shift();
            }
        }
        t += groups * U;
    }
#pragma unroll 1
    for (; t < end; ++t) careful(t);
    N zero[H];
#pragma unroll
    for (int h = 0; h < H; ++h) fill(zero[h], 0.f);
    dx = static_cast<XT*>(A.dx) + (long long)p.b * A.T * A.C + p.c;
#pragma unroll 1
    for (t = max(t0, te); t < t1; ++t) store<XT, V>(dx, (long long)t * A.C, zero);  // behind the end
    if (!A.parts) return;
    float* out = A.parts + ((long long)p.b * A.runs + p.run) * (K + 1) * A.C + p.c;
#pragma unroll
    for (int k = 0; k < K; ++k) store<float, V>(out, (long long)k * A.C, dw[k]);
    store<float, V>(out, (long long)K * A.C, db);
}

// Column sums of [n][(K+1) C]: 32 columns and 32 slices of the rows per CTA, slices added up in order.
inline __global__ void __launch_bounds__(1024) weights_kernel(const ConvArgs A, long long n) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long cols = (long long)(A.K + 1) * A.C, c = (long long)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < cols)
#pragma unroll 4
        for (long long i = slice; i < n; i += 32) t += A.parts[i * cols + c];
    sum[slice][lane] = t;
    __syncthreads();
    if (slice || c >= cols) return;
    for (int s = 1; s < 32; ++s) t += sum[s][lane];
    const int k = (int)(c / A.C), ch = (int)(c - (long long)k * A.C);
    if (k < A.K) {
        if (A.dw) A.dw[(long long)ch * A.K + k] = t;
    } else if (A.dbias) {
        A.dbias[ch] = t;
    }
}

}  // namespace conv
}  // namespace lattice

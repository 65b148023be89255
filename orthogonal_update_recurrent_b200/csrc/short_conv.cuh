// short_conv.cuh -- short causal convolution of every channel over the tokens of a sequence, its
// backward pass and its single-token step (sm_100a).
//
//   v_t = bias + sum_k w[k] x_{t-K+1+k},  y_t = act(v_t);  x before the first token: the state, or 0
// Backward, with e_t = dy_t act'(v_t):
//   dx_s = sum_j w[K-1-j] e_{s+j},  dw[k] = sum_t e_t x_{t-K+1+k},  dbias = sum_t e_t
//
// HBM bounds it: x is read once and y written once. A thread has V neighbouring channels and
// walks down a run of tokens with the last K-1 inputs in registers, loads of U tokens under way at
// once; a run's K-1 first inputs are its neighbour's last ones and mostly come from the L2.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};
template <class T, int V>
__device__ __forceinline__ Vec<T, V> load(const void* p, long long i) {
    return *reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(p) + i);
}
template <class T, int V>
__device__ __forceinline__ void store(void* p, long long i, const float* f) {
    Vec<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) put(r.v[v], f[v]);
    *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(p) + i) = r;
}
template <class T, int V>
__device__ __forceinline__ void values(const Vec<T, V>& r, float* f) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = to_f(r.v[v]);
}
template <class T, int V>
__device__ __forceinline__ Vec<T, V> zeros() {
    Vec<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) put(r.v[v], 0.f);
    return r;
}
template <class XT>
__device__ __forceinline__ float weight(const ConvArgs& A, const void* p, long long i) {
    return sizeof(XT) == 4 || A.w32 ? static_cast<const float*>(p)[i] : to_f(static_cast<const XT*>(p)[i]);
}
// A thread's weights, from the oldest input's on, and bias
template <class XT, int K, int V>
__device__ __forceinline__ void weights(const ConvArgs& A, int c, float (*w)[V], float* bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][v] = weight<XT>(A, A.w, (long long)(c + v) * K + k);
        bias[v] = A.bias ? weight<XT>(A, A.bias, c + v) : 0.f;
    }
}
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-1.442695041f * v)); }

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
__global__ void __launch_bounds__(256) fwd_kernel(const ConvArgs A) {
    constexpr int U = 8;
    const Place<V> p(A);
    if (!p.in) return;
    float w[K][V], bias[V], win[K][V];  // win[k]: x_{t-K+1+k}
    weights<XT, K, V>(A, p.c, w, bias);
    const int t0 = p.run * A.run, t1 = min(A.T, t0 + A.run), te = min(t1, p.len);
    Vec<XT, V> last[K > 1 ? K - 1 : 1];
    if (p.run == 0 && A.state_out) {  // read before anything is written: the state may be updated in place
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j] = input<XT, K, V>(A, p.b, p.c, p.len - (K - 1) + j);
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (t0 < te) values<XT, V>(input<XT, K, V>(A, p.b, p.c, t0 - (K - 1) + k), win[k]);
    }
    const long long xat = p.b * A.xbs + p.c, yat = (long long)p.b * A.T * A.C + p.c;
    for (int tb = t0; tb < te; tb += U) {
        Vec<XT, V> r[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (tb + j < te) r[j] = load<XT, V>(A.x, xat + (tb + j) * A.xts);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (tb + j >= te) break;
            values<XT, V>(r[j], win[K - 1]);
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = bias[v];
#pragma unroll
                for (int k = 0; k < K; ++k) s = fmaf(w[k][v], win[k][v], s);
                y[v] = A.silu ? s * sigmoid(s) : s;
#pragma unroll
                for (int k = 0; k < K - 1; ++k) win[k][v] = win[k + 1][v];
            }
            store<XT, V>(A.y, yat + (long long)(tb + j) * A.C, y);
        }
    }
    const float none[V] = {};
    for (int t = max(t0, te); t < t1; ++t) store<XT, V>(A.y, yat + (long long)t * A.C, none);  // behind the end
    if (p.run == 0 && A.state_out) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<Vec<XT, V>*>(static_cast<XT*>(A.state_out) + ((long long)p.b * (K - 1) + j) * A.C + p.c) = last[j];
    }
}

// One token: the state's rows move up by one
template <class XT, int K, int V>
__global__ void __launch_bounds__(256) step_kernel(const ConvArgs A) {
    const Place<V> p(A);
    if (!p.in) return;
    float w[K][V], bias[V], x[V], y[V];
    Vec<XT, V> r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) r[k] = input<XT, K, V>(A, p.b, p.c, k - (K - 1));
    weights<XT, K, V>(A, p.c, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = bias[v];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        values<XT, V>(r[k], x);
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = fmaf(w[k][v], x[v], y[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = A.silu ? y[v] * sigmoid(y[v]) : y[v];
    store<XT, V>(A.y, (long long)p.b * A.C + p.c, y);
#pragma unroll
    for (int k = 1; k < K; ++k)
        *reinterpret_cast<Vec<XT, V>*>(static_cast<XT*>(A.state_out) + ((long long)p.b * (K - 1) + k - 1) * A.C + p.c) = r[k];
}

// A run's dx needs e of the K-1 tokens behind it, whose own inputs reach K-1 tokens back: x and dy of 2 (K-1)
// and K-1 tokens are read twice. The weights' gradients are summed over the run and written as
// one row [C][K+1] of the workspace per run.
template <class XT, int K, int V>
__global__ void __launch_bounds__(256) bwd_kernel(const ConvArgs A) {
    constexpr int U = 4;
    const Place<V> p(A);
    if (!p.in) return;
    float w[K][V], bias[V], win[K][V], e[K][V] = {}, dw[K][V] = {}, db[V] = {};  // e[j]: e_{t-K+1+j}
    weights<XT, K, V>(A, p.c, w, bias);
    const int t0 = p.run * A.run, t1 = min(A.T, t0 + A.run), te = min(t1, p.len);
    const long long xat = p.b * A.xbs + p.c, gat = p.b * A.ybs + p.c, oat = (long long)p.b * A.T * A.C + p.c;
    // what the final state's cotangent adds to input row s
    auto state_part = [&](int s, float* f) {
        const int j = s - (p.len - (K - 1));
        if (!A.dstate_out || j < 0 || s >= p.len) return;
        float d[V];
        values<XT, V>(load<XT, V>(A.dstate_out, ((long long)p.b * (K - 1) + j) * A.C + p.c), d);
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] += d[v];
    };
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        if (t0 < te) values<XT, V>(input<XT, K, V>(A, p.b, p.c, t0 - (K - 1) + k), win[k]);
    const bool head = p.run == 0 && A.dstate;  // writes the gradients of the rows before the first token
    const int end = t0 < te || head ? te + K - 1 : t0;
    for (int tb = t0; tb < end; tb += U) {
        Vec<XT, V> rx[U], rg[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (tb + j < min(end, p.len)) rx[j] = load<XT, V>(A.x, xat + (tb + j) * A.xts), rg[j] = load<XT, V>(A.dy, gat + (tb + j) * A.yts);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int t = tb + j;
            if (t >= end) break;
            if (t < p.len) {
                values<XT, V>(rx[j], win[K - 1]);
                values<XT, V>(rg[j], e[K - 1]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (A.silu) {
                        float s = bias[v];
#pragma unroll
                        for (int k = 0; k < K; ++k) s = fmaf(w[k][v], win[k][v], s);
                        const float q = sigmoid(s);
                        e[K - 1][v] *= fmaf(s * q, 1.f - q, q);
                    }
                }
                if (t < te) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += e[K - 1][v];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][v] = fmaf(e[K - 1][v], win[k][v], dw[k][v]);
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) e[K - 1][v] = 0.f;
            }
            const int s = t - (K - 1);
            if (s >= t0 || head) {
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) d[v] = fmaf(w[K - 1 - k][v], e[k][v], d[v]);
                }
                state_part(s, d);
                if (s >= t0) store<XT, V>(A.dx, oat + (long long)s * A.C, d);
                else store<XT, V>(A.dstate, ((long long)p.b * (K - 1) + K - 1 + s) * A.C + p.c, d);
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v], e[k][v] = e[k + 1][v];
        }
    }
    const float none[V] = {};
    for (int t = max(t0, te); t < t1; ++t) store<XT, V>(A.dx, oat + (long long)t * A.C, none);
    if (!A.parts) return;
    float* out = A.parts + ((long long)p.b * A.runs + p.run) * (K + 1) * A.C + p.c;  // [K+1][C]
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) out[(long long)k * A.C + v] = k < K ? dw[k < K ? k : 0][v] : db[v];
}

// Column sums of [n][(K+1) C]: 32 columns and 32 slices of the rows per CTA, slices added up in order.
inline __global__ void __launch_bounds__(1024) weights_kernel(const ConvArgs A, int n) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long cols = (long long)(A.K + 1) * A.C, c = (long long)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int i = slice; i < n; i += 32) t += A.parts[i * cols + c];
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

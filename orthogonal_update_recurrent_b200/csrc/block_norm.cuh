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
// stay in registers between its sums, and what is left is to keep enough bytes in flight.
// A thread has 8 elements of a row. A row of up to 256 elements takes a part of a warp and
// its sums are shuffles, one of up to 8192 (read one by one: 6144; backward, with twice the
// registers: 4096) a CTA, a longer one a cluster of 2 or 4 CTAs.
// CTAs stay and take rows by turns: each loads its next row before it works on the one it
// has, and its threads keep their columns' weights, and the sums of the weights' gradients,
// in shared memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "args.h"
#include "f32x2.cuh"
#include "waits.cuh"

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

// The gates' activations and, if wanted, their derivatives. The normal distribution function
// of gelu is formula 7.1.26 of Abramowitz and Stegun's Handbook (absolute error 7.5e-8
// here), whose exponential the derivative needs too.
template <bool SLOPE>
__device__ __forceinline__ void activate(int act, F2 g, F2& f, F2& df) {
    if (act == kGelu) {
        const F2 x = each(g, [](float v) { return fabsf(v); });
        const F2 e = each(mul2(mul2(g, g), f2(-0.72134752f)), ex2);  // exp(-g^2/2)
        const F2 t = each(fma2(x, f2(0.3275911f * 0.70710678f), f2(1.f)), rcp);
        F2 p = f2(1.061405429f * 0.5f);
        p = fma2(p, t, f2(-1.453152027f * 0.5f));
        p = fma2(p, t, f2(1.421413741f * 0.5f));
        p = fma2(p, t, f2(-0.284496736f * 0.5f));
        p = fma2(p, t, f2(0.254829592f * 0.5f));
        const F2 tail = mul2(mul2(p, t), e), head = fma2(tail, f2(-1.f), f2(1.f));
        float g0, g1, t0, t1, h0, h1;
        parts(g, g0, g1), parts(tail, t0, t1), parts(head, h0, h1);
        const F2 cdf = f2(g0 >= 0.f ? h0 : t0, g1 >= 0.f ? h1 : t1);
        f = mul2(g, cdf);
        if constexpr (SLOPE) df = fma2(mul2(g, f2(0.39894228f)), e, cdf);
    } else {
        const F2 s = each(each(mul2(g, f2(-1.442695041f)), [](float n) { return 1.f + ex2(n); }), rcp);
        f = act == kSilu ? mul2(g, s) : s;
        if constexpr (SLOPE) {
            const F2 q = fma2(s, f2(-1.f), f2(1.f));
            df = act == kSilu ? mul2(s, fma2(g, q, f2(1.f))) : mul2(s, q);
        }
    }
}

// A row's threads: tpr lanes of a warp (SUB), or a CTA, or the CTAs of a cluster.
// Sums over them: shuffles, one barrier per sum in a CTA (buffers by turns), and in a
// cluster an asynchronous store of the CTA's sum to every CTA, counted on its mbarrier.
template <bool SUB>
struct RowSums {
    float* red;               // [2][256]
    float4* box;              // [2][4][2]: the CTAs' sums
    uint32_t bars;
    volatile uint32_t* abort;
    int K, rank, tpr, k;      // k: sums so far
    __device__ __forceinline__ RowSums(const NormArgs& A) : K(SUB ? 1 : A.K), rank(SUB ? 0 : blockIdx.x % A.K), tpr(A.tpr), k(0) {
        __shared__ float red_[2 * 256];
        __shared__ float4 box_[2 * 8];
        __shared__ __align__(8) uint64_t bars_[2];
        __shared__ uint32_t abort_;
        red = red_, box = box_, bars = ptx::smem_u32(bars_), abort = &abort_;
        if (K > 1) {
            if (threadIdx.x == 0) {
                ptx::mbar_init(bars, 1);
                ptx::mbar_init(bars + 8, 1);
                abort_ = 0u;
                ptx::fence_mbar_init();
            }
            sync_cluster();  // nobody sends before every CTA's mbarriers stand
        }
    }
    static __device__ __forceinline__ void sync_cluster() {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __device__ __forceinline__ void end() const {  // nobody leaves while something may be on its way to it
        if (K > 1) sync_cluster();
    }
    // Sums of M <= 8 values over the row's threads, in every thread. More than two values:
    // a lane hands half of them on at each of the first steps (8 values in 9 shuffles
    // instead of 40) and ends with one value's sum over its warp.
    template <int M>
    __device__ __forceinline__ void sum(float* v) {
        constexpr unsigned ALL = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        if constexpr (M <= 2) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (!SUB || o < tpr)
#pragma unroll
                    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(ALL, v[m], o);
            if constexpr (SUB) return;
        } else if (SUB && tpr < 8) {
            for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(ALL, v[m], o);
            return;
        }
        float own = 0.f;  // M > 2: the lane's value
        int mine = 0;     // and which
        if constexpr (M > 2) {
            float t[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) t[m] = m < M ? v[m] : 0.f;
            int o = SUB ? tpr >> 1 : 16;
            const int o1 = o;
#pragma unroll
            for (int n = 4; n > 0; n >>= 1, o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int m = 0; m < n; ++m) {
                    const float keep = up ? t[m + n] : t[m], give = up ? t[m] : t[m + n];
                    t[m] = keep + __shfl_xor_sync(ALL, give, o);
                }
                mine += up ? n : 0;
            }
            own = t[0];
#pragma unroll
            for (int k_ = 0; k_ < 2; ++k_, o >>= 1)
                if (o > 0) own += __shfl_xor_sync(ALL, own, o);
            if constexpr (SUB) {  // value m stands with the lane whose bits below tpr spell it
                const int base = lane & ~(tpr - 1);
#pragma unroll
                for (int m = 0; m < M; ++m)
                    v[m] = __shfl_sync(ALL, own, base + (m & 4 ? o1 : 0) + (m & 2 ? o1 >> 1 : 0) + (m & 1 ? o1 >> 2 : 0));
                return;
            }
        }
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5, buf = k & 1;
        float* r = red + buf * 256;  // [warp][8], M <= 2: [m][warp]
        if constexpr (M <= 2) {
            if (lane == 0)
#pragma unroll
                for (int m = 0; m < M; ++m) r[m * 32 + warp] = v[m];
        } else if ((lane & 3) == 0) {
            r[warp * 8 + mine] = own;
        }
        __syncthreads();
        if constexpr (M <= 2) {
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] = lane < nw ? r[m * 32 + lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(ALL, v[m], o);
        } else {
            own = 0.f;  // lane: value lane % 8 of every fourth warp
            for (int w = lane >> 3; w < nw; w += 4) own += r[w * 8 + (lane & 7)];
            own += __shfl_xor_sync(ALL, own, 8);
            own += __shfl_xor_sync(ALL, own, 16);
            if (K == 1)
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] = __shfl_sync(ALL, own, m);
        }
        if (K > 1) {
            float4* b = box + buf * 8;  // [rank][2]
            if constexpr (M <= 2) {
                if ((int)threadIdx.x < K)
                    ptx::st_async_v4(ptx::mapa(ptx::smem_u32(b + rank * 2), threadIdx.x),
                                     make_float4(v[0], M > 1 ? v[M - 1] : 0.f, 0.f, 0.f), ptx::mapa(bars + 8 * buf, threadIdx.x));
            } else if (warp == 0) {
                float4 a;
                const int q = lane & 4;  // lane 0..K-1: values 0-3 to CTA lane; 4 + 0..K-1: values 4-7
                a.x = __shfl_sync(ALL, own, q), a.y = __shfl_sync(ALL, own, q + 1);
                a.z = __shfl_sync(ALL, own, q + 2), a.w = __shfl_sync(ALL, own, q + 3);
                if (lane < 8 && (lane & 3) < K)
                    ptx::st_async_v4(ptx::mapa(ptx::smem_u32(b + rank * 2 + (lane >> 2)), lane & 3), a,
                                     ptx::mapa(bars + 8 * buf, lane & 3));
            }
            if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(bars + 8 * buf, K * (M <= 2 ? 16 : 32));
            tc_wait(bars + 8 * buf, (k >> 1) & 1, abort);
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] = 0.f;
            for (int q = 0; q < K; ++q) {
                const float4 a = b[q * 2], d = b[q * 2 + 1];
                const float t[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += t[m];
            }
        }
        ++k;
    }
};

// How a thread reads its 8 columns of a row: one by one, tpr apart; as a vector; or as a vector
// that starts up to 7 columns before the row does. The last is for widths that are no
// multiple of 8: row i starts m = i D mod 8 elements past a multiple of 16 bytes, and the grid's
// step is a multiple of 8 rows (of 8/gcd(D, 8)), so that m, and with it a thread's columns, are
// the same in all its rows. Only a row's two outer vectors, the edges, have columns of other
// rows: they are put to 0 after the load and left out of the store (bf16, one by one and
// so: 16384 rows of 2055, both norms, forward 106 and 66 us, backward 262 and 223 us; 8192 rows of
// 6055 with a gate, 117 and 86 us, 442 and 209 us).
constexpr int kOdd = kNormOdd, kVec = kNormVec, kShift = kNormShift;

template <int MODE>
struct Columns {
    static constexpr int V = MODE == kOdd ? 1 : 8, NV = 8 / V;
    int first, step, D;
    __device__ __forceinline__ Columns(const NormArgs& A, int rank, int tid, unsigned row)
        : first(rank * A.tpr * 8 + tid * V - (MODE == kShift ? (int)(row * (unsigned)A.D & 7u) : 0)), step(A.tpr), D(A.D) {}
    __device__ __forceinline__ int at(int j) const { return first + j * step; }
    __device__ __forceinline__ bool has(int j) const { return at(j) < D; }
    __device__ __forceinline__ bool edge() const { return MODE == kShift && (first < 0 || first + 8 > D); }
    __device__ __forceinline__ bool mine(int v) const { return (unsigned)(first + v) < (unsigned)D; }  // the vector's v-th
};
// `inside`: the row's outer vectors lie within the array, too
template <class XT, int MODE>
__device__ __forceinline__ void load8(Raw<XT, Columns<MODE>::V>* r, const void* p, bool f32, long long row,
                                      const Columns<MODE>& c, bool inside = true) {
    constexpr int V = Columns<MODE>::V;
    if (MODE == kShift && !inside && c.edge()) {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if (!c.mine(v)) continue;
            const Raw<XT, 1> e = load<XT, 1>(p, f32, row + c.first + v);
            if (sizeof(XT) == 4 || f32) r[0].w[v % V] = e.w[0];
            else r[0].w[v / 2 % V] = v & 1 ? (r[0].w[v / 2 % V] & 0xffffu) | e.w[0] << 16 : e.w[0];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < Columns<MODE>::NV; ++j)
        if (c.has(j)) r[j] = load<XT, V>(p, f32, row + c.at(j));
}
// Puts the columns of other rows to 0.
template <class XT, int MODE>
__device__ __forceinline__ void trim8(Raw<XT, Columns<MODE>::V>* r, bool f32, const Columns<MODE>& c) {
    if constexpr (MODE == kShift) {
        if (!c.edge()) return;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if (c.mine(v)) continue;
            if (sizeof(XT) == 4 || f32) r[0].w[v] = 0u;
            else r[0].w[v / 2] &= v & 1 ? 0xffffu : 0xffff0000u;
        }
    }
}
// The 8 values as four pairs.
template <class XT, int V>
__device__ __forceinline__ void values8(const Raw<XT, V>* r, bool f32, F2* f) {
    if (sizeof(XT) == 4 || f32) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            f[v] = f2(__uint_as_float(r[2 * v / V].w[2 * v % V]), __uint_as_float(r[(2 * v + 1) / V].w[(2 * v + 1) % V]));
    } else if constexpr (sizeof(XT) == 2) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float a, b, other;
            if constexpr (V == 8) {
                unpack(XT(), r[0].w[v], a, b);
            } else {
                unpack(XT(), r[2 * v].w[0], a, other);
                unpack(XT(), r[2 * v + 1].w[0], b, other);
            }
            f[v] = f2(a, b);
        }
    }
}
template <class XT, int MODE>
__device__ __forceinline__ void store8(void* p, bool f32, long long row, const Columns<MODE>& c, const F2* q) {
    constexpr int V = Columns<MODE>::V;
    float f[8];
#pragma unroll
    for (int v = 0; v < 4; ++v) parts(q[v], f[2 * v], f[2 * v + 1]);
    if (c.edge()) {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            if (c.mine(v)) store<XT, 1>(p, f32, row + c.first + v, f + v);
        return;
    }
#pragma unroll
    for (int j = 0; j < Columns<MODE>::NV; ++j)
        if (c.has(j)) store<XT, V>(p, f32, row + c.at(j), f + j * V);
}
__device__ __forceinline__ float both(F2 a) {
    float x, y;
    parts(a, x, y);
    return x + y;
}
// Sum of the products of 8 values.
__device__ __forceinline__ float dot8(const F2* a, const F2* b) {
    F2 t = mul2(a[0], b[0]);
#pragma unroll
    for (int v = 1; v < 4; ++v) t = fma2(a[v], b[v], t);
    return both(t);
}
// 8 floats of the thread's own in shared memory, [2][threads] of 16 bytes
__device__ __forceinline__ void own_read(const ulonglong2* p, F2* f) {
    const ulonglong2 a = p[threadIdx.x], b = p[blockDim.x + threadIdx.x];
    f[0].v = a.x, f[1].v = a.y, f[2].v = b.x, f[3].v = b.y;
}
__device__ __forceinline__ void own_write(ulonglong2* p, const F2* f) {
    p[threadIdx.x] = make_ulonglong2(f[0].v, f[1].v);
    p[blockDim.x + threadIdx.x] = make_ulonglong2(f[2].v, f[3].v);
}
// The columns' weights into the thread's shared memory: w_post with the scale, w_pre. Columns
// past the row's end have weight 0, and their values stay 0 all the way.
template <class XT, int MODE>
__device__ __forceinline__ void keep_weights(const NormArgs& A, const Columns<MODE>& c, ulonglong2* wq, ulonglong2* wp) {
    constexpr int V = Columns<MODE>::V;
    Raw<XT, V> raw[8 / V] = {};
    F2 f[4];
    for (int k = 0; k < 2; ++k) {
        const void* w = k ? A.w_pre : A.w_post;
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = f2(1.f);
        if (w) {
            if constexpr (MODE == kShift) {
                float t[8];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    t[v] = 0.f;
                    if (c.mine(v)) values<XT, 1>(load<XT, 1>(w, A.w32, c.first + v), A.w32, t + v);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] = f2(t[2 * v], t[2 * v + 1]);
            } else {
                load8<XT, MODE>(raw, w, A.w32, 0, c);
                values8<XT, V>(raw, A.w32, f);
            }
        }
        if (!k)
#pragma unroll
            for (int v = 0; v < 4; ++v) f[v] = mul2(f[v], f2(A.scale));
        own_write(k ? wp : wq, f);
    }
}
// Where row i of a strided array starts: groups of A.G rows, contiguous within a group.
struct RowAt {
    unsigned grp, off;
    __device__ __forceinline__ RowAt(const NormArgs& A, unsigned i) : grp(A.G == 1 ? i : i / A.G), off(0) {
        off = A.G == 1 ? 0u : i - grp * A.G;
    }
    __device__ __forceinline__ long long in(const NormArgs& A, unsigned stride) const {
        return (long long)((unsigned long long)grp * stride + (unsigned long long)off * (unsigned)A.D);
    }
};

// Types of a call beside its own XT, and its parts. Y32; R32: y; residual, r and dr are fp32.
// PRE: with the norm before the next block (-1: the call says). As run-time flags, types alone
// cost the backward pass 20 of 71 instructions per element.
template <class XT_, int MODE_, bool GATE_, bool Y32_, bool R32_, int PRE_>
struct Form {
    using XT = XT_;
    static constexpr int MODE = MODE_, V = MODE == kOdd ? 1 : 8;
    static constexpr bool GATE = GATE_;
    static constexpr bool Y32 = Y32_, R32 = R32_;
    static __device__ __forceinline__ bool pre(bool runtime) { return PRE_ < 0 ? runtime : PRE_ == 1; }
};

// Threads of a CTA at most: 64 registers each forward (80 where rows are read element by
// element), 128 backward.
constexpr int kFwdThreads = 1024, kFwdOddThreads = 768, kBwdThreads = 512;

template <class F, bool SUB>
__global__ void __launch_bounds__(SUB ? 256 : F::V == 8 ? kFwdThreads : kFwdOddThreads, SUB ? (F::V == 8 ? 4 : 2) : 1)
norm_fwd_kernel(const NormArgs A) {
    using XT = typename F::XT;
    constexpr int MODE = F::MODE, V = F::V, NV = 8 / V;
    constexpr bool GATE = F::GATE;
    constexpr bool y32 = F::Y32, r32 = F::R32;
    const bool pre = F::pre(A.n_out != nullptr);
    extern __shared__ __align__(16) ulonglong2 own[];
    ulonglong2 *wq = own, *wp = own + 2 * blockDim.x;
    RowSums<SUB> sums(A);
    const int tid = SUB ? threadIdx.x % A.tpr : threadIdx.x;
    const unsigned rows = SUB ? blockDim.x / A.tpr : 1, lane_row = SUB ? threadIdx.x / A.tpr : 0;
    const unsigned row0 = blockIdx.x / sums.K * rows;
    const Columns<MODE> c(A, sums.rank, tid, row0 + lane_row);
    keep_weights<XT, MODE>(A, c, wq, wp);
    const unsigned N = (unsigned)A.N, step = gridDim.x / sums.K * rows;
    Raw<XT, V> ry[NV] = {}, rg[NV] = {}, rr[NV] = {};
    auto fetch = [&](unsigned i) {
        if (i >= N) return;
        const RowAt at(A, i);
        const bool inside = i + 8 < N;  // the rows behind it hold a vector's columns past its end
        load8<XT, MODE>(ry, A.y, y32, at.in(A, A.ys), c, inside);
        if constexpr (GATE) load8<XT, MODE>(rg, A.gate, false, at.in(A, A.gs), c, inside);
        if (A.residual) load8<XT, MODE>(rr, A.residual, r32, at.in(A, A.rs), c, inside);
    };
    unsigned first = row0;
    fetch(first + lane_row);
    for (; first < N; first += step) {  // N + step + rows < 2^32
        const unsigned i = first + lane_row;
        const bool in = i < N;
        F2 y[4], r[4], g[4], w[4];
        trim8<XT, MODE>(ry, y32, c);
        values8<XT, V>(ry, y32, y);
        if constexpr (GATE) {
            trim8<XT, MODE>(rg, false, c);
            values8<XT, V>(rg, false, g);
        }
        if (A.residual) {
            trim8<XT, MODE>(rr, r32, c);
            values8<XT, V>(rr, r32, r);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) r[v] = f2(0.f);
        }
        fetch(i + step);  // the next row's values are on their way during this row's sums
        own_read(wq, w);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if constexpr (GATE) {
                F2 f, df;
                activate<false>(A.act, g[v], f, df);
                w[v] = mul2(w[v], f);
            }
        float s[1], rho = 1.f;
        if (A.post) {
            s[0] = dot8(y, y);
            sums.template sum<1>(s);
            rho = rsqrtf(fmaf(s[0], A.inv_d, A.eps));
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) r[v] = fma2(mul2(y[v], f2(rho)), w[v], r[v]);
        if (in) store8<XT, MODE>(A.r_out, r32, (long long)i * A.D, c, r);
        if (pre) {
            s[0] = dot8(r, r);
            own_read(wp, w);
            sums.template sum<1>(s);
            rho = rsqrtf(fmaf(s[0], A.inv_d, A.eps));
#pragma unroll
            for (int v = 0; v < 4; ++v) r[v] = mul2(mul2(r[v], f2(rho)), w[v]);
            if (in) store8<XT, MODE>(A.n_out, false, (long long)i * A.D, c, r);
        }
    }
    sums.end();
}

// The weights' gradients: the CTA's sums (dq, dp: 8 floats of each thread's own columns) to its row of the
// workspace, added up by norm_dw_kernel.
template <class XT, int MODE, bool SUB>
__device__ __forceinline__ void write_parts(const NormArgs& A, const Columns<MODE>& c, const ulonglong2* dq, const ulonglong2* dp,
                                            unsigned rows, unsigned row0, int K) {
    if (!A.parts) return;
    float* out = A.parts + (long long)(blockIdx.x / K) * 2 * A.D;
    __syncthreads();
    if constexpr (MODE == kShift) {
        for (int k = 0; k < 2; ++k) {
            const float* p = reinterpret_cast<const float*>(k ? dp : dq);
            if constexpr (SUB) {  // a column is another thread's in each of the rows
                for (int q = threadIdx.x; q < A.D; q += blockDim.x) {
                    float t = 0.f;
                    for (unsigned i = 0; i < rows; ++i) {
                        const unsigned j = q + ((row0 + i) * (unsigned)A.D & 7u), v = j & 7u;
                        t += p[((v >> 2) * blockDim.x + i * A.tpr + (j >> 3)) * 4 + (v & 3u)];
                    }
                    out[k * A.D + q] = t;
                }
            } else {
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    if (c.mine(v)) out[k * A.D + c.first + v] = p[((v >> 2) * blockDim.x + threadIdx.x) * 4 + (v & 3)];
            }
        }
        return;
    }
    if (SUB && (int)threadIdx.x >= A.tpr) return;
    for (int k = 0; k < 2; ++k) {
        const ulonglong2* p = k ? dp : dq;
        F2 t[4];
        own_read(p, t);
        for (unsigned q = 1; q < rows; ++q) {  // a CTA's rows side by side, one by one
            const ulonglong2 a = p[q * A.tpr + threadIdx.x], b = p[blockDim.x + q * A.tpr + threadIdx.x];
            t[0] = add2(t[0], F2{a.x}), t[1] = add2(t[1], F2{a.y}), t[2] = add2(t[2], F2{b.x}), t[3] = add2(t[3], F2{b.y});
        }
        store8<float, MODE>(out, true, k * A.D, c, t);
    }
}

// With t = scale y w_post act(gate), v = rho1 t, m = w_pre dn and e as above, the sum for dy
//   sum(du y) = sum(e t) = sum(dr t) + rho2 sum(m t) - k sum(r t), k = rho2^3 mean(m r),
// is taken apart, so that it needs no exchange of its own after e is known.
template <class F, bool SUB>
__global__ void __launch_bounds__(SUB ? 256 : kBwdThreads, SUB ? 2 : 1) norm_bwd_kernel(const NormArgs A) {
    using XT = typename F::XT;
    constexpr int MODE = F::MODE, V = F::V, NV = 8 / V;
    constexpr bool GATE = F::GATE;
    constexpr bool y32 = F::Y32, r32 = F::R32;
    const bool pre = F::pre(A.dn != nullptr);
    extern __shared__ __align__(16) ulonglong2 own[];
    ulonglong2 *wq = own, *wp = own + 2 * blockDim.x, *dq = own + 4 * blockDim.x, *dp = own + 6 * blockDim.x;
    RowSums<SUB> sums(A);
    const int tid = SUB ? threadIdx.x % A.tpr : threadIdx.x;
    const unsigned rows = SUB ? blockDim.x / A.tpr : 1, lane_row = SUB ? threadIdx.x / A.tpr : 0;
    const unsigned row0 = blockIdx.x / sums.K * rows;
    const Columns<MODE> c(A, sums.rank, tid, row0 + lane_row);
    keep_weights<XT, MODE>(A, c, wq, wp);
    {
        const F2 zero[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
        own_write(dq, zero);
        own_write(dp, zero);
    }
    const unsigned N = (unsigned)A.N, step = gridDim.x / sums.K * rows;
    Raw<XT, V> ry[NV] = {}, rg[NV] = {}, rr[NV] = {}, rd[NV] = {}, rn[NV] = {};
    auto fetch = [&](unsigned i) {
        if (i >= N) return;
        const RowAt at(A, i);
        const bool inside = i + 8 < N;  // the rows behind it hold a vector's columns past its end
        load8<XT, MODE>(ry, A.y, y32, at.in(A, A.ys), c, inside);
        if constexpr (GATE) load8<XT, MODE>(rg, A.gate, false, at.in(A, A.gs), c, inside);
        if (A.dr) load8<XT, MODE>(rd, A.dr, r32, at.in(A, A.drs), c, inside);
        if (pre) {
            if (A.residual) load8<XT, MODE>(rr, A.residual, r32, at.in(A, A.rs), c, inside);
            load8<XT, MODE>(rn, A.dn, false, at.in(A, A.dns), c, inside);
        }
    };
    unsigned first = row0;
    fetch(first + lane_row);
    for (; first < N; first += step) {
        const unsigned i = first + lane_row;
        const bool in = i < N;
        const long long o = (long long)i * A.D;
        F2 y[4], e[4], r[4], m[4], f[4], df[4], t[4], w[4], acc[4];
        trim8<XT, MODE>(ry, y32, c);
        values8<XT, V>(ry, y32, y);
        if constexpr (GATE) {
            trim8<XT, MODE>(rg, false, c);
            values8<XT, V>(rg, false, f);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) e[v] = r[v] = f2(0.f);
        if (A.dr) {
            trim8<XT, MODE>(rd, r32, c);
            values8<XT, V>(rd, r32, e);
        }
        if (pre) {
            if (A.residual) {
                trim8<XT, MODE>(rr, r32, c);
                values8<XT, V>(rr, r32, r);
            }
            trim8<XT, MODE>(rn, false, c);
            values8<XT, V>(rn, false, m);
        }
        if (SUB && first + rows > N && !in) {  // the last turn's rows past the end count as 0
#pragma unroll
            for (int v = 0; v < 4; ++v) y[v] = e[v] = r[v] = m[v] = f[v] = f2(0.f);
        }
        fetch(i + step);  // the next row's values are on their way during this row's sums
        float s[5], rho1 = 1.f, k = 0.f;
        s[0] = dot8(y, y);
        own_read(wq, w);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if constexpr (GATE) activate<true>(A.act, f[v], f[v], df[v]);
            t[v] = mul2(y[v], w[v]);
            if constexpr (GATE) t[v] = mul2(t[v], f[v]);
        }
        if (!pre && A.post) {
            s[1] = dot8(e, t);
            sums.template sum<2>(s);
            k = s[1];
        } else if (A.post) {
            sums.template sum<1>(s);
        }
        if (A.post) rho1 = rsqrtf(fmaf(s[0], A.inv_d, A.eps));
        if (pre) {
            own_read(dp, acc);
            own_read(wp, w);
            F2 dnr[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                r[v] = fma2(t[v], f2(rho1), r[v]);
                dnr[v] = mul2(m[v], r[v]);
                m[v] = mul2(m[v], w[v]);
            }
            s[0] = dot8(r, r), s[1] = dot8(m, r);
            if (A.post) {
                s[2] = dot8(e, t), s[3] = dot8(m, t), s[4] = dot8(r, t);
                sums.template sum<5>(s);
            } else {
                sums.template sum<2>(s);
            }
            // from the sum on: rho^3 alone leaves fp32's range for rows of 1e13 and an eps of 1e-26
            const float rho2 = rsqrtf(fmaf(s[0], A.inv_d, A.eps)), k2 = s[1] * A.inv_d * rho2 * rho2 * rho2;
            if (A.post) k = fmaf(rho2, s[3], s[2]) - k2 * s[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                acc[v] = fma2(dnr[v], f2(rho2), acc[v]);
                e[v] = fma2(r[v], f2(-k2), fma2(m[v], f2(rho2), e[v]));
            }
            own_write(dp, acc);
        }
        if (A.dresidual && in) store8<XT, MODE>(A.dresidual, r32, o, c, e);
        k *= -rho1 * A.inv_d * rho1;  // and once more with y
        own_read(wq, w);
        own_read(dq, acc);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            e[v] = mul2(e[v], f2(rho1));
            const F2 u = mul2(e[v], y[v]);
            acc[v] = GATE ? fma2(u, f[v], acc[v]) : add2(u, acc[v]);
            if constexpr (GATE) df[v] = mul2(mul2(df[v], u), w[v]);
            e[v] = mul2(e[v], GATE ? mul2(w[v], f[v]) : w[v]);
            e[v] = fma2(mul2(y[v], f2(rho1)), f2(k), e[v]);
        }
        own_write(dq, acc);
        if constexpr (GATE)
            if (in) store8<XT, MODE>(A.dgate, false, o, c, df);
        if (in) store8<XT, MODE>(A.dy, y32, o, c, e);
    }
    sums.end();
    write_parts<XT, MODE, SUB>(A, c, dq, dp, rows, row0, sums.K);
}

// dw = scale (w_post) or 1 (w_pre) times the column sums of [parts][2 D]: 32 columns and
// SLICES slices of the rows per CTA, slices added up in order.
template <int SLICES>
__global__ void __launch_bounds__(SLICES * 32) norm_dw_kernel(const float* parts, int nparts, int D, float scale, float* dw_post,
                                                      float* dw_pre) {
    __shared__ float sum[SLICES][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * D)
#pragma unroll 8
        for (int i = slice; i < nparts; i += SLICES) t += parts[(long long)i * 2 * D + c];
    sum[slice][lane] = t;
    __syncthreads();
    if (slice || c >= 2 * D) return;
    for (int s = 1; s < SLICES; ++s) t += sum[s][lane];
    if (c < D) {
        if (dw_post) dw_post[c] = t * scale;
    } else if (dw_pre) {
        dw_pre[c - D] = t;
    }
}

}  // namespace norm
}  // namespace lattice

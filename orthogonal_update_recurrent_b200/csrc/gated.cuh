// gated.cuh -- gated linear recurrence over whole sequences, its backward pass and its
// single-token step (sm_100a).
//
// Per (batch, channel), channel = (head, element):
//   h_t = a_t h_{t-1} + s(a_t) x_t,  y_t = h_t
// with the gate a = z (value) or a = sigmoid(z)^tau (logit) and the write scale
// s = 1 (plain), 1 - a (leaky) or sqrt(max(0, 1 - a^2)) (unit). z has one entry per channel
// or one per head.
//
// Every element is used once per direction, so HBM bounds all three kernels; the time
// axis is what has to be parallel. A warp takes a run of R consecutive tokens of 32 V
// channels and reduces it to the pair (P, H) with h_out = P h_in + H. The pairs of a CTA's
// NW warps are exchanged through shared memory, those of a cluster's K CTAs (K consecutive
// tiles of NW*R tokens) through distributed shared memory; each warp folds the pairs before
// its own, in token order, onto the state that entered the iteration, and completes its
// run. Every fold has a fixed order: results do not change from run to run.
//
// Inputs are staged a few iterations ahead in shared memory by cp.async, each warp the rows
// of its own runs, so that a stage needs no barrier and the loads never wait for the
// exchange.
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
namespace gated {

constexpr int kValue = 0, kLogit = 1, kLogitTau = 2;  // gate forms (kLogit: tau = 1)
constexpr int kPlain = 0, kLeaky = 1, kUnit = 2;      // write forms
constexpr int kZSame = 0, kZ32 = 1, kZHead = 2;       // z per channel in x's type or fp32; per head

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// V consecutive elements at p (n of them inside the row); VEC: one vector access.
template <bool VEC, class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p, int n) {
    if constexpr (VEC) {
        return *reinterpret_cast<const Vec<T, V>*>(p);
    } else {
        Vec<T, V> r;
#pragma unroll
        for (int v = 0; v < V; ++v) r.v[v] = v < n ? p[v] : from_f<T>(0.f);
        return r;
    }
}
template <bool VEC, class T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* f, int n) {
    if constexpr (VEC) {
        Vec<T, V> r;
        if constexpr (sizeof(T) == 2 && V % 2 == 0) {  // two at a time: one conversion instruction
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                if constexpr (std::is_same<T, __half>::value)
                    *reinterpret_cast<__half2*>(&r.v[v]) = __floats2half2_rn(f[v], f[v + 1]);
                else
                    *reinterpret_cast<__nv_bfloat162*>(&r.v[v]) = __floats2bfloat162_rn(f[v], f[v + 1]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) r.v[v] = from_f<T>(f[v]);
        }
        *reinterpret_cast<Vec<T, V>*>(p) = r;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < n) p[v] = from_f<T>(f[v]);
    }
}

constexpr float kLog2e = 1.442695041f;

// exp(w) - 1 for -0.25 <= w <= 0 by the power series.
constexpr float kSmall = -0.25f;
__device__ __forceinline__ F2 expm1_small(F2 w) {
    F2 p = f2(1.f / 720.f);
    p = fma2(p, w, f2(1.f / 120.f));
    p = fma2(p, w, f2(1.f / 24.f));
    p = fma2(p, w, f2(1.f / 6.f));
    p = fma2(p, w, f2(0.5f));
    return fma2(mul2(w, w), p, w);
}

// The gates a and q = 1 - a of two channels. Errors of a gate near 1 are multiplied by the
// retention time, so its last bit must not be biased, as an approximate reciprocal's may
// be: with t = exp(-z), r = 1/(1 + t) gets one Newton step, a = r (2 - (1 + t) r), and 1 - a is
// t a, which keeps its relative accuracy however near 1 a is. exp(-z) stops at 2^126. With
// tau, `fast` says that the warp's gates of the token have no z < 0 and tau <= 1, which leaves out what those need
// (65536 tokens of 2048 channels, tau 1/8, unit write: 264 us, 317 us without `fast`; by log(1 + t)
// and exp, for every z, 307 us).
template <int GATE>
__device__ __forceinline__ void gates_of(F2 z, const GatedArgs& A, bool fast, F2& a, F2& q) {
    if constexpr (GATE == kValue) {
        a = z;
        q = fma2(z, f2(-1.f), f2(1.f));
    } else if constexpr (GATE == kLogit) {
        const F2 t = each(mul2(z, f2(-kLog2e)), [](float n) { return ex2(min_nan(n, 126.f)); });
        const F2 nd = fma2(t, f2(-1.f), f2(-1.f));  // -(1 + t)
        const F2 r = each(nd, rcp);                 // -1/(1 + t)
        a = mul2(r, fma2(nd, r, f2(-2.f)));
        q = mul2(t, a);
        a = add2(a, f2(-1.17549435e-38f));  // 2^-126 at z = -inf becomes the 0 it stands for
    } else {
        // With t = exp(-|z|) <= 1, q0 = 1 - (1 + t)^-tau is t times a polynomial for tau <= 1; a
        // larger tau halves it often enough and squares 1 - q0 as often. z < 0 has the factor
        // exp(tau z) besides. Every element's result depends on its own z alone.
        const F2 t = each(z, [](float v) { return ex2(-fabsf(v) * kLog2e); });
        F2 p = {A.poly[kGatedPoly - 1]};
#pragma unroll
        for (int k = kGatedPoly - 2; k >= 0; --k) p = fma2(p, t, F2{A.poly[k]});
        q = mul2(p, t);
        a = fma2(q, f2(-1.f), f2(1.f));
        if (fast) return;
        for (int k = 0; k < A.squares; ++k) {
            q = mul2(q, fma2(q, f2(-1.f), f2(2.f)));
            a = mul2(a, a);
        }
        const F2 x = mul2(f2(A.tau), each(z, [](float v) { return fminf(v, 0.f); }));
        const F2 e = each(mul2(x, f2(kLog2e)), ex2), m = expm1_small(x), e1 = add2(e, f2(-1.f));
        float x0, x1, m0, m1, e10, e11;
        parts(x, x0, x1), parts(m, m0, m1), parts(e1, e10, e11);
        const F2 em = f2(x0 > kSmall ? m0 : e10, x1 > kSmall ? m1 : e11);
        q = fma2(mul2(a, f2(-1.f)), em, q);
        // near 1: 1 - (1 - a), one rounding
        const F2 near = fma2(q, f2(-1.f), f2(1.f)), far = mul2(a, e);
        float q0, q1, n0, n1, f0, f1;
        parts(q, q0, q1), parts(near, n0, n1), parts(far, f0, f1);
        a = f2(q0 < 0.5f ? n0 : f0, q1 < 0.5f ? n1 : f1);
    }
}
// da/dz
template <int GATE>
__device__ __forceinline__ F2 slopes_of(F2 z, float tau, F2 a, F2 q) {
    if constexpr (GATE == kLogit) return mul2(a, q);
    const F2 s = each(z, [](float v) {  // sigmoid(-z)
        const float t = ex2(-fabsf(v) * kLog2e);
        return (v >= 0.f ? t : 1.f) * rcp(1.f + t);
    });
    return mul2(mul2(f2(tau), a), s);
}
template <int GATE, int WRITE>
__device__ __forceinline__ F2 writes_of(F2 a, F2 q) {
    if constexpr (WRITE == kPlain) return f2(1.f);
    if constexpr (WRITE == kLeaky) return q;
    const F2 v = mul2(q, add2(a, f2(1.f)));
    return each(v, [](float x) { return root(GATE == kValue ? max_nan(x, 0.f) : x); });
}
// ds/da of the unit write, 0 where s = 0
__device__ __forceinline__ F2 unit_slopes(F2 a, F2 s) {
    float a0, a1, s0, s1;
    parts(a, a0, a1), parts(s, s0, s1);
    return f2(s0 > 0.f ? -a0 * rcp(s0) : 0.f, s1 > 0.f ? -a1 * rcp(s1) : 0.f);
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The exchange of a cluster's pairs: every CTA sends its own to all K, into one of two
// buffers by turns, as asynchronous stores that count their bytes on the receiver's
// mbarrier, so that neither side fences its other memory traffic (a cluster barrier's
// release waited for the rows' stores: 65536 tokens of 2048 channels, tau 1, took 203 us with
// one, 185 us so). A buffer is sent to again only after its sender has everyone's pairs of the
// iteration between, and a CTA sends those after its warps have read the buffer.
struct Exchange {
    uint32_t bars;  // two mbarriers
    volatile uint32_t* abort;
    uint32_t bytes;
    __device__ __forceinline__ Exchange(uint64_t* b, volatile uint32_t* a, int nbytes, bool cluster) {
        bars = ptx::smem_u32(b);
        abort = a;
        bytes = (uint32_t)nbytes;
        if (!cluster) return;
        if (threadIdx.x == 0) {
            ptx::mbar_init(bars, 1);
            ptx::mbar_init(bars + 8, 1);
            *abort = 0u;
            ptx::fence_mbar_init();
        }
        cluster_sync_all();  // nobody sends before every CTA's mbarriers stand
        if (threadIdx.x == 0) {
            ptx::mbar_arrive_expect_tx(bars, bytes);
            ptx::mbar_arrive_expect_tx(bars + 8, bytes);
        }
    }
    // N floats (a multiple of 4) to the same shared-memory place of CTA `rank`
    template <int N>
    __device__ __forceinline__ void send(const float* local, int rank, int buf, const float* f) const {
        const uint32_t bar = ptx::mapa(bars + 8 * buf, rank), at = ptx::mapa(ptx::smem_u32(local), rank);
#pragma unroll
        for (int v = 0; v < N; v += 4) ptx::st_async_v4(at + 4 * v, make_float4(f[v], f[v + 1], f[v + 2], f[v + 3]), bar);
    }
    // Everyone's pairs of the buffer's turn-th use. A wait that gives up sets the status
    // word; the ones after it do not wait, so the kernel runs to its end.
    __device__ __forceinline__ void wait(int buf, int turn) const {
        tc_wait(bars + 8 * buf, (uint32_t)turn & 1u, abort);
        if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(bars + 8 * buf, bytes);
    }
};

__device__ __forceinline__ int row_length(const GatedArgs& A, int b) {
    if (!A.lengths) return A.T;
    const int n = A.lengths[b];
    return n < 0 ? 0 : n > A.T ? A.T : n;
}

// How rows start: at any element (kAny), at a multiple of a lane's V channels (kPairs), or of 16
// bytes (kWide). Shifted rows stand in a stage as far behind a multiple of 16 bytes as in memory,
// and have room for it.
constexpr int kAny = 0, kPairs = 1, kWide = 2;
template <int ROWS, class T>
constexpr bool kShifted = ROWS == kAny || (ROWS == kPairs && sizeof(T) == 4);
template <int ROWS, class T, int V>
struct RowOf {
    static constexpr int N = 32 * V, STRIDE = N + (kShifted<ROWS, T> ? 16 / (int)sizeof(T) : 0);
};
// Copies a run's R rows of 32 V channels (n of them exist from the tile's first on) into a
// stage of the warp's, and moves on to the warp's next run. kWide: 16 bytes at a time. 16-bit
// kPairs: a lane's V channels. Shifted rows: the 16-byte pieces that a row's bytes lie in, the
// last one as far as the row goes. 8 sequences of 4096 tokens, forward and backward: 2047
// channels in bf16 331 and 498 us with elements loaded one by one, 140 and 332 us with shifted
// pieces; 2046 channels in bf16 102 and 190 us by lanes, 111 and 212 us with shifted
// pieces, in fp32 220 and 375 us by lanes, 160 and 296 us with shifted pieces. Where few
// channels leave the device idle it can be the other way: 37 channels in bf16, one sequence of
// 32768 tokens, backward, 156 us one by one, 201 us with shifted pieces.
template <int ROWS, class T, int V, int R>
struct Stager {
    static constexpr int ROW = 32 * V, PER = 16 / sizeof(T), CH = ROW / PER, STEP = 32 / CH;  // chunks per row
    static constexpr int STRIDE = RowOf<ROWS, T, V>::STRIDE;
    static_assert(CH <= 32 && R % STEP == 0 && R <= 32, "whole warps of chunks, a lane per row");
    const T* p;            // of the next run: the lane's first row, or its first piece there
    long long ts, move;    // STEP rows, by lanes: one; from run to run
    uintptr_t back;        // bytes from the run's first row to the lane's
    uintptr_t lowest;      // the array's first byte: nothing before it is read
    long long row;         // bytes from row to row
    int n;                 // shifted: a row's bytes; else whether the lane copies
    __device__ __forceinline__ Stager(const void* array, const T* base, long long token_stride, int channels, long long first,
                                      long long ahead, int lane)
        : ts(STEP * token_stride), move(ahead * token_stride), lowest(reinterpret_cast<uintptr_t>(array)),
          row(token_stride * (long long)sizeof(T)) {
        p = base + (first + lane / CH) * token_stride;
        back = (uintptr_t)(lane / CH * row);
        n = (channels < ROW ? channels : ROW) * (int)sizeof(T);
        if constexpr (ROWS == kWide) {
            p += lane % CH * PER;
            n = lane % CH * PER < channels;
        } else if constexpr (!kShifted<ROWS, T>) {
            p = base + first * token_stride + lane * V;
            ts = token_stride;
            n = lane * V < channels;
        }
    }
    __device__ __forceinline__ void copy(T* stage, int rows, int lane) {
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(stage);
        const T* q = p;
        if constexpr (ROWS == kWide) {
            if (!n) return;
#pragma unroll
            for (int k = 0; k < R / STEP; ++k) {
                if (rows >= R || k * STEP + lane / CH < rows)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + (k * 32 + lane) * 16), "l"(q) : "memory");
                q += ts;
            }
        } else if constexpr (!kShifted<ROWS, T>) {
            if (!n) return;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r < rows)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d + (r * ROW + lane * V) * (int)sizeof(T)), "l"(q),
                                 "n"(V * sizeof(T))
                                 : "memory");
                q += ts;
            }
        } else {
#pragma unroll
            for (int k = 0; k < R / STEP; ++k) {
                part(stage, d, reinterpret_cast<uintptr_t>(q), k * STEP + lane / CH, lane % CH, rows);
                q += ts;
            }
            if (lane < R) part(stage, d, reinterpret_cast<uintptr_t>(p) - back + lane * row, lane, CH, rows);
        }
    }
    // Piece k of the row at a
    __device__ __forceinline__ void part(T* stage, uint32_t d, uintptr_t a, int row, int k, int rows) const {
        const uintptr_t src = (a & ~(uintptr_t)15) + 16 * k;
        const int left = n - 16 * k + (int)(a & 15);  // bytes of the row, from src on
        if (row >= rows || left <= 0) return;
        if (src >= lowest) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + (uint32_t)(row * STRIDE * (int)sizeof(T) + 16 * k)),
                         "l"(src), "r"(left < 16 ? left : 16)
                         : "memory");
        } else {  // the array starts within these 16 bytes
            T* e = stage + row * STRIDE;
            for (int v = 0; v < PER; ++v) {
                const uintptr_t s = src + v * sizeof(T);
                if (s >= a && s < a + n) e[v] = *reinterpret_cast<const T*>(s);
            }
        }
    }
};
// Where a run's rows start in their stages, behind a multiple of 16 bytes.
template <int ROWS, class T>
struct RowStart {
    uint32_t at, step;
    __device__ __forceinline__ RowStart(const T* base, long long token_stride)
        : at((uint32_t)reinterpret_cast<uintptr_t>(base)), step((uint32_t)(token_stride * sizeof(T))) {}
    __device__ __forceinline__ const T* row(const T* stage, int stride, int t0, int r) const {
        if constexpr (!kShifted<ROWS, T>) return stage + r * stride;
        else return stage + r * stride + ((at + (uint32_t)(t0 + r) * step & 15u) / sizeof(T));
    }
};
// Rows behind the sequence's end are made neutral in the stage: a gate of 1 that writes 0.
template <int GATE>
__device__ __forceinline__ float neutral_z() {
    return GATE == kValue ? 1.f : __int_as_float(0x7f800000);
}
template <class T, int STRIDE, int R>
__device__ __forceinline__ void fill_rows(T* stage, int first, float value, int lane) {
    for (int i = (first > 0 ? first : 0) * STRIDE + lane; i < R * STRIDE; i += 32) stage[i] = from_f<T>(value);
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}
// N pairs of channels at p
template <class T, int N>
__device__ __forceinline__ void read_pairs(const T* p, F2* f) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int v = 0; v < N; v += 2) {
                const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + 2 * v);
                f[v].v = t.x, f[v + 1].v = t.y;
            }
        } else {
#pragma unroll
            for (int v = 0; v < N; ++v) f[v].v = *reinterpret_cast<const unsigned long long*>(p + 2 * v);
        }
    } else {
        const Vec<uint32_t, N> w = *reinterpret_cast<const Vec<uint32_t, N>*>(p);
#pragma unroll
        for (int v = 0; v < N; ++v) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w.v[v]));
                f[v] = f2(t.x, t.y);
            } else {
                f[v] = f2(__uint_as_float(w.v[v] << 16), __uint_as_float(w.v[v] & 0xffff0000u));
            }
        }
    }
}
// A row's, wherever it starts
template <int ROWS, class T, int N>
__device__ __forceinline__ void read_row(const T* p, F2* f) {
    if constexpr (!kShifted<ROWS, T> || (ROWS == kPairs && N == 1)) {
        read_pairs<T, N>(p, f);
    } else if constexpr (ROWS == kPairs) {
#pragma unroll
        for (int v = 0; v < N; ++v) read_pairs<T, 1>(p + 2 * v, f + v);
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v) f[v] = f2(to_f(p[2 * v]), to_f(p[2 * v + 1]));
    }
}
// The same for fp32 shared memory, and back
template <int N>
__device__ __forceinline__ void write_pairs(float* p, const F2* f) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int v = 0; v < N; v += 2) *reinterpret_cast<ulonglong2*>(p + 2 * v) = make_ulonglong2(f[v].v, f[v + 1].v);
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v) *reinterpret_cast<unsigned long long*>(p + 2 * v) = f[v].v;
    }
}
template <bool VEC, class T, int N>
__device__ __forceinline__ void store_pairs(T* p, const F2* f, int n) {
    float t[2 * N];
#pragma unroll
    for (int v = 0; v < N; ++v) parts(f[v], t[2 * v], t[2 * v + 1]);
    store_vec<VEC, T, 2 * N>(p, t, n);
}
// A row of a result by the whole warp, n of the lane's channels (lanes without any call too). Two
// 16-bit channels per lane that start on an odd element are stored as the words that they
// share with the lane before.
template <bool VEC, class T, int N>
__device__ __forceinline__ void store_row(T* p, const F2* f, int n, int lane) {
    if constexpr (VEC || sizeof(T) == 4 || N != 1) {
        if (n > 0) store_pairs<VEC, T, N>(p, f, n);
    } else {
        Vec<T, 2> own;
        float a, b;
        parts(f[0], a, b);
        own.v[0] = from_f<T>(a), own.v[1] = from_f<T>(b);
        if ((reinterpret_cast<uintptr_t>(p) & 2u) == 0) {  // the same in all lanes
            if (n >= 2) *reinterpret_cast<Vec<T, 2>*>(p) = own;
            else if (n == 1) p[0] = own.v[0];
        } else {
            uint32_t w;
            memcpy(&w, &own, 4);
            const uint32_t before = __shfl_up_sync(0xffffffffu, w, 1);
            if (n >= 1) {
                if (lane == 0) p[0] = own.v[0];
                else *reinterpret_cast<uint32_t*>(p - 1) = before >> 16 | w << 16;
                if (n >= 2 && (lane == 31 || n == 2)) p[1] = own.v[1];
            }
        }
    }
}
template <bool VEC, int N>
__device__ __forceinline__ void load_state(const float* p, int n, F2* f) {  // p may be null: 0
#pragma unroll
    for (int v = 0; v < N; ++v) f[v] = f2(0.f);
    if (p && n > 0) {
        const Vec<float, 2 * N> t = load_vec<VEC, float, 2 * N>(p, n);
#pragma unroll
        for (int v = 0; v < N; ++v) f[v] = f2(t.v[2 * v], t.v[2 * v + 1]);
    }
}
// The sign bits of a lane's z of a row, at any place of the words.
template <int ROWS, class ZT, int N>
__device__ __forceinline__ uint32_t signs(const ZT* p) {
    constexpr int W = N * 2 * sizeof(ZT) / 4;
    uint32_t bits = 0;
    if constexpr (!kShifted<ROWS, ZT>) {
        const Vec<uint32_t, W> w = *reinterpret_cast<const Vec<uint32_t, W>*>(p);
#pragma unroll
        for (int v = 0; v < W; ++v) bits |= w.v[v];
    } else if constexpr (sizeof(ZT) == 4) {
#pragma unroll
        for (int v = 0; v < W; ++v) bits |= reinterpret_cast<const uint32_t*>(p)[v];
    } else {
#pragma unroll
        for (int v = 0; v < 2 * N; ++v) bits |= reinterpret_cast<const uint16_t*>(p)[v];
    }
    return bits & (sizeof(ZT) == 4 ? 0x80000000u : 0x80008000u);
}
// The rows of a run, as bits, in which some lane's z is negative; mostly none.
template <int ROWS, class ZT, int N, int R>
__device__ __forceinline__ uint32_t negative_rows(const RowStart<ROWS, ZT>& at, const ZT* z, int stride, int t0) {
    uint32_t all = 0, rows = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) all |= signs<ROWS, ZT, N>(at.row(z, stride, t0, r));
    if (!__any_sync(0xffffffffu, all != 0)) return 0;
#pragma unroll
    for (int r = 0; r < R; ++r) rows |= signs<ROWS, ZT, N>(at.row(z, stride, t0, r)) ? 1u << r : 0u;
    return __reduce_or_sync(0xffffffffu, rows);
}
template <class XT>
__device__ __forceinline__ float load_gate(const void* z, long long off, bool z32) {
    if (sizeof(XT) == 4 || z32) return static_cast<const float*>(z)[off];
    return to_f(static_cast<const XT*>(z)[off]);
}

// Gates per head: a warp's R tokens have R * nh of them, nh heads in its channels. Lane i
// works out gates i, i + 32, ... (gate = token * nh + head) and leaves the W values that
// each token needs in the warp's shared memory, every value twice, ready for packed
// arithmetic. The raw gates are staged with the rows: a register that a load is still to
// fill cannot be moved on, which kept them one iteration ahead and made the load's latency
// the iteration's length (head gates of the mid-size layer 84 us, staged 61 us, 54 us since).
template <class XT, int V, int R, int W>
struct HeadGates {
    static constexpr int PER = V * R / 16;           // gates per lane: at most 32 V / 16 heads
    static constexpr int BYTES = R * 2 * V * W * 8;  // of a warp
    int shift, j;    // log2 nh; which head the lane's channels have
    long long base;  // of the warp's first head
    int heads;       // of them that exist
    int parity;      // of the first head's place, where 16-bit gates are copied as whole words
    float z[(PER + 1) / 2 * 2] = {};
    __device__ __forceinline__ HeadGates(const GatedArgs& A, int b, int c0, int lane) {
        const int nh = 32 * V / A.d > 0 ? 32 * V / A.d : 1;  // d is a power of two
        shift = 31 - __clz(nh);
        j = lane * V / A.d;
        base = (long long)b * A.zbs + c0 / A.d;
        heads = (A.C - c0 + A.d - 1) / A.d;
        parity = c0 / A.d;
    }
    static constexpr int STAGE = PER * 128;  // bytes of a warp's stage: a word a gate
    __device__ __forceinline__ void stage(const GatedArgs& A, uint32_t* words, int t0, int len, int lane) const {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = k * 32 + lane, r = i >> shift, hd = i - (r << shift);
            if (r < R && t0 + r < len && hd < heads) {
                const long long off = base + (t0 + r) * A.zts + hd;
                if (sizeof(XT) == 4 || A.z32 || A.zwords) {
                    const uint32_t* p = static_cast<const uint32_t*>(A.z) + (sizeof(XT) == 4 || A.z32 ? off : off >> 1);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(words + i)),
                                 "l"(p)
                                 : "memory");
                } else {
                    words[i] = static_cast<const uint16_t*>(A.z)[off];
                }
            }
        }
    }
    __device__ __forceinline__ void read(const GatedArgs& A, const uint32_t* words, int t0, int len, float neutral, int lane) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = k * 32 + lane, r = i >> shift, hd = i - (r << shift);
            z[k] = neutral;
            if (r < R && t0 + r < len && hd < heads) {
                const uint32_t w = words[i];
                if (sizeof(XT) == 4 || A.z32) {
                    z[k] = __uint_as_float(w);
                } else {
                    const uint16_t h = (uint16_t)(A.zwords && ((parity + hd) & 1) ? w >> 16 : w);
                    XT t;
                    memcpy(&t, &h, 2);
                    z[k] = to_f(t);
                }
            }
        }
    }
    // f(pair of z, out[W])
    template <class F>
    __device__ __forceinline__ void keep(float* mine, int lane, F f) {
#pragma unroll
        for (int k = 0; k < PER; k += 2) {
            if (k && (R << shift) <= k * 32) break;
            F2 out[W];
            f(f2(z[k], z[k + 1]), out);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int i = (k + m) * 32 + lane;
                if (k + m < PER && i < (R << shift)) {
                    F2 twice[W];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float lo, hi;
                        parts(out[w], lo, hi);
                        twice[w] = f2(m ? hi : lo);
                    }
                    write_pairs<W>(mine + i * 2 * W, twice);
                }
            }
        }
        __syncwarp();
    }
    // f(m, token, head, pair of z) for each of the lane's gates, z its m-th of the pair
    template <class F>
    __device__ __forceinline__ void each_gate(F f, int lane) const {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = k * 32 + lane, r = i >> shift, hd = i - (r << shift);
            if (r < R && hd < heads) f(k & 1, r, hd, f2(z[k & ~1], z[k | 1]));
        }
    }
    // token r's first M values for the lane's channels
    template <int M>
    __device__ __forceinline__ void get(const float* mine, int r, F2* out) const {
        read_pairs<float, M>(mine + ((r << shift) + j) * 2 * W, out);
    }
};

// ---- forward
template <class XT, int ZM, int ROWS, int V, int R, int NW, int NST>
struct FwdLayout {
    using ZT = typename std::conditional<ZM == kZ32, float, XT>::type;
    static constexpr int XROW = RowOf<ROWS, XT, V>::STRIDE, ZROW = RowOf<ROWS, ZT, V>::STRIDE;
    static constexpr int HO = ZM == kZHead && V > 2 ? 4 : V, PAIR = (HO + V + 3) / 4 * 4;  // floats of a lane's (P, H)
    static constexpr int X = R * XROW * sizeof(XT), Z = ZM == kZHead ? V * R * 8 : R * ZROW * sizeof(ZT);
    static constexpr int STAGE = X + Z;                      // bytes of a warp's stage
    static constexpr int HG = NW * NST * STAGE;              // a warp's gates per head
    static constexpr int SW = HG + (ZM == kZHead ? NW * HeadGates<XT, V, R, 2>::BYTES : 0);  // [2][NW][32][PAIR]
    static constexpr int SB = SW + 2 * NW * 32 * PAIR * 4;   // a cluster's mbarriers and abort flag
    static constexpr int SC = SB + 32;                       // [2][K][32][PAIR]; one CTA: [2][32][V], the state
    static constexpr int bytes(int K) { return SC + 2 * 32 * 4 * (K > 1 ? K * PAIR : V); }
};

// A lane has N = V/2 pairs of channels; with one gate per head, its first pair of gates
// holds the same gate twice.
template <class XT, int ZM, int FORM, int ROWS, int V, int R, int NW, int NST, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB) gated_fwd_kernel(const GatedArgs A) {
    using Lay = FwdLayout<XT, ZM, ROWS, V, R, NW, NST>;
    using ZT = typename Lay::ZT;
    constexpr int GATE = FORM / 3, WRITE = FORM % 3, L = NW * R, PAIR = Lay::PAIR, HO = Lay::HO, N = V / 2;
    constexpr bool HEAD = ZM == kZHead, VEC = ROWS != kAny;
    constexpr int NG = HEAD ? 1 : N;
    static_assert(kGatedMark % R == 0 || R % kGatedMark == 0, "runs and marks fall together");
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sw = reinterpret_cast<float*>(smem + Lay::SW) + lane * PAIR;
    float* sc = reinterpret_cast<float*>(smem + Lay::SC);
    const int K = A.K, rank = blockIdx.x % K;
    const int ct = (blockIdx.x / K) % A.ctiles, b = blockIdx.x / K / A.ctiles;
    const int c0 = ct * 32 * V, c = c0 + lane * V, n = A.C - c;  // the lane's channels: n of them exist
    const bool on = n > 0;
    const XT* x = static_cast<const XT*>(A.x) + (long long)b * A.xbs + c0;
    const ZT* z = static_cast<const ZT*>(A.z) + (long long)b * A.zbs + c0;
    XT* y = static_cast<XT*>(A.y) + (long long)b * A.T * A.C + c;
    const int len = row_length(A, b);
    const int iters = (len + K * L - 1) / (K * L);

    F2 h[N];  // one CTA: the last warp's; a cluster: everyone's
    load_state<VEC, N>(A.h0 ? A.h0 + (long long)b * A.C + c : nullptr, n, h);
    if (K == 1 && warp == NW - 1) write_pairs<N>(sc + lane * V, h);

    Exchange ex(reinterpret_cast<uint64_t*>(smem + Lay::SB), reinterpret_cast<volatile uint32_t*>(smem + Lay::SB + 16),
                K * 32 * PAIR * 4, K > 1);
    unsigned char* mine = smem + warp * NST * Lay::STAGE;
    int ts = rank * L + warp * R;  // the run that is staged next
    Stager<ROWS, XT, V, R> sx(A.x, x, A.xts, A.C - c0, ts, K * L, lane);
    Stager<ROWS, ZT, V, R> sz(A.z, z, A.zts, A.C - c0, HEAD ? 0 : ts, K * L, lane);
    const RowStart<ROWS, XT> x_at(x, A.xts);
    const RowStart<ROWS, ZT> z_at(z, A.zts);
    HeadGates<XT, V, R, 2> hg(A, b, c0, lane);
    auto stage = [&](int slot) {
        if (ts < len) {
            unsigned char* s = mine + slot * Lay::STAGE;
            sx.copy(reinterpret_cast<XT*>(s), len - ts, lane);
            sx.p += sx.move;
            if constexpr (HEAD) {
                hg.stage(A, reinterpret_cast<uint32_t*>(s + Lay::X), ts, len, lane);
            } else {
                sz.copy(reinterpret_cast<ZT*>(s + Lay::X), len - ts, lane);
                sz.p += sz.move;
            }
            ts += K * L;
        }
        stage_commit();
    };
    float* gates = reinterpret_cast<float*>(smem + Lay::HG) + warp * (HeadGates<XT, V, R, 2>::BYTES / 4);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) stage(s);
    int slot = 0;
    for (int it = 0; it < iters; ++it) {
        const int t0 = (it * K + rank) * L + warp * R, buf = it & 1;
        stage(slot == 0 ? NST - 1 : slot - 1);
        stage_wait<NST - 1>();
        XT* xw = reinterpret_cast<XT*>(mine + slot * Lay::STAGE);
        ZT* zw = reinterpret_cast<ZT*>(mine + slot * Lay::STAGE + Lay::X);
        const XT* xs = xw + lane * V;
        const ZT* zs = zw + lane * V;
        slot = slot == NST - 1 ? 0 : slot + 1;
        const bool full = t0 + R <= len;
        if (!full) {
            fill_rows<XT, Lay::XROW, R>(xw, len - t0, 0.f, lane);
            if constexpr (!HEAD) fill_rows<ZT, Lay::ZROW, R>(zw, len - t0, neutral_z<GATE>(), lane);
            __syncwarp();
        }
        if constexpr (HEAD) {
            hg.read(A, reinterpret_cast<const uint32_t*>(zw), t0, len, neutral_z<GATE>(), lane);
            hg.keep(gates, lane, [&](F2 hz, F2* out) {
                F2 hq;
                gates_of<GATE>(hz, A, false, out[0], hq);
                out[1] = writes_of<GATE, WRITE>(out[0], hq);
            });
        }
        uint32_t slow = ~0u;  // rows of which some gate needs more
        if constexpr (!HEAD && GATE == kLogitTau)
            if (A.squares == 0) slow = negative_rows<ROWS, ZT, N, R>(z_at, zs, Lay::ZROW, t0);
        // P: products of the run's gates, H: the run's states from h = 0, after each token
        F2 P[R][NG], H[R][N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            F2 xf[N], zf[N], a[N], w[N];
            read_row<ROWS, XT, N>(x_at.row(xs, Lay::XROW, t0, r), xf);
            if constexpr (HEAD) {
                F2 t[2];
                hg.template get<2>(gates, r, t);
                a[0] = t[0], w[0] = t[1];
            } else {
                read_row<ROWS, ZT, N>(z_at.row(zs, Lay::ZROW, t0, r), zf);
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int k = HEAD ? 0 : v;
                if constexpr (!HEAD) {
                    F2 q;
                    gates_of<GATE>(zf[v], A, !(slow >> r & 1u), a[v], q);
                    w[v] = writes_of<GATE, WRITE>(a[v], q);
                }
                const F2 u = WRITE == kPlain ? xf[v] : mul2(w[k], xf[v]);
                H[r][v] = r ? fma2(a[k], H[r ? r - 1 : 0][v], u) : u;
                if (v < NG) P[r][k] = r ? mul2(P[r ? r - 1 : 0][k], a[k]) : a[k];
            }
        }
        {
            float* p = sw + (buf * NW + warp) * 32 * PAIR;
            write_pairs<NG>(p, P[R - 1]);
            write_pairs<N>(p + HO, H[R - 1]);
        }
        __syncthreads();
        F2 hin[N];
        auto fold = [&](const float* p, F2* state) {
            F2 p_[NG], h_[N];
            read_pairs<float, NG>(p, p_);
            read_pairs<float, N>(p + HO, h_);
#pragma unroll
            for (int v = 0; v < N; ++v) state[v] = fma2(p_[HEAD ? 0 : v], state[v], h_[v]);
        };
        if (K == 1) {
            read_pairs<float, N>(sc + (buf * 32 + lane) * V, hin);
        } else {
            if (warp < K) {  // each warp sends the CTA's pair to one CTA of the cluster
                F2 p_[NG], h_[N];
#pragma unroll
                for (int v = 0; v < NG; ++v) p_[v] = f2(1.f);
#pragma unroll
                for (int v = 0; v < N; ++v) h_[v] = f2(0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float* p = sw + (buf * NW + w) * 32 * PAIR;
                    F2 t[NG];
                    fold(p, h_);
                    read_pairs<float, NG>(p, t);
#pragma unroll
                    for (int v = 0; v < NG; ++v) p_[v] = mul2(p_[v], t[v]);
                }
                float f[PAIR] = {};
#pragma unroll
                for (int v = 0; v < NG; ++v) parts(p_[v], f[2 * v], f[2 * v + 1]);
#pragma unroll
                for (int v = 0; v < N; ++v) parts(h_[v], f[HO + 2 * v], f[HO + 2 * v + 1]);
                for (int q = warp; q < K; q += NW) ex.send<PAIR>(sc + ((buf * K + rank) * 32 + lane) * PAIR, q, buf, f);
            }
            ex.wait(buf, it >> 1);
            for (int q = 0; q < K; ++q) {
                if (q == rank) {
#pragma unroll
                    for (int v = 0; v < N; ++v) hin[v] = h[v];
                }
                fold(sc + ((buf * K + q) * 32 + lane) * PAIR, h);
            }
        }
        for (int w = 0; w < warp; ++w) fold(sw + (buf * NW + w) * 32 * PAIR, hin);
        if (K == 1 && warp == NW - 1) {
#pragma unroll
            for (int v = 0; v < N; ++v) h[v] = fma2(P[R - 1][HEAD ? 0 : v], hin[v], H[R - 1][v]);
            write_pairs<N>(sc + ((buf ^ 1) * 32 + lane) * V, h);
        }
        if (on || !VEC) {  // a row's store may be the whole warp's
            if (on && A.marks) {
#pragma unroll
                for (int r = 0; r < R; r += kGatedMark) {
                    F2 f[N];
#pragma unroll
                    for (int v = 0; v < N; ++v) f[v] = r ? fma2(P[r ? r - 1 : 0][HEAD ? 0 : v], hin[v], H[r ? r - 1 : 0][v]) : hin[v];
                    if (t0 % kGatedMark == 0 && t0 + r < len)
                        store_pairs<VEC, float, N>(A.marks + ((long long)b * A.nmarks + (t0 + r) / kGatedMark) * A.C + c, f, n);
                }
            }
            if (A.y) {
                XT* yt = y + (long long)t0 * A.C;
                auto put = [&](int r) {
                    F2 f[N];
#pragma unroll
                    for (int v = 0; v < N; ++v) f[v] = fma2(P[r][HEAD ? 0 : v], hin[v], H[r][v]);
                    store_row<VEC, XT, N>(yt + (long long)r * A.C, f, n, lane);
                };
                if (full) {
#pragma unroll
                    for (int r = 0; r < R; ++r) put(r);
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (t0 + r < len) put(r);
                }
            }
        }
    }
    if (K > 1) cluster_sync_all();  // nobody leaves while something may be on its way to it
    if (!on) return;
    if (A.h_out && rank == 0 && warp == NW - 1) store_pairs<VEC, float, N>(A.h_out + (long long)b * A.C + c, h, n);
    if (A.y) {  // rows behind the sequence's end
        const float zero[V] = {};
        for (int t = len + rank * NW + warp; t < A.T; t += K * NW) store_vec<VEC, XT, V>(y + (long long)t * A.C, zero, n);
    }
}

// ---- backward
// With g_t = dy_t + a_{t+1} g_{t+1} (g_len += dh_T): dx = s g, dz = (da/dz) g (h_{t-1} + x ds/da),
// dh_0 = a_1 g_1. Tiles run from the sequence's end to its start; a run's
// states are rebuilt from the mark that the forward pass left at its start, and the
// adjoint enters from behind, by the runs' pairs (P, G).
template <class XT, int ZM, int ROWS, int V, int R, int NW, int NST>
struct BwdLayout {
    using ZT = typename std::conditional<ZM == kZ32, float, XT>::type;
    static constexpr int XROW = RowOf<ROWS, XT, V>::STRIDE, ZROW = RowOf<ROWS, ZT, V>::STRIDE;
    static constexpr int HO = ZM == kZHead ? 4 : V, PAIR = (HO + V + 3) / 4 * 4;  // floats of a lane's (P, G)
    static constexpr int X = R * XROW * sizeof(XT), Z = ZM == kZHead ? V * R * 8 : R * ZROW * sizeof(ZT);
    static constexpr int M = 2 * X + Z;           // the mark's place in a stage
    static constexpr int STAGE = M + 32 * V * 4;
    static constexpr int HG = NW * NST * STAGE;             // a warp's gates per head
    static constexpr int SW = HG + (ZM == kZHead ? NW * HeadGates<XT, V, R, 4>::BYTES : 0);  // [2][NW][32][PAIR]
    static constexpr int SB = SW + 2 * NW * 32 * PAIR * 4;  // a cluster's mbarriers and abort flag
    static constexpr int SC = SB + 32;                      // [2][K][32][PAIR]; one CTA: [2][32][V], the adjoint
    static constexpr int bytes(int K) { return SC + 2 * 32 * 4 * (K > 1 ? K * PAIR : V); }
};

template <class XT, int ZM, int FORM, int ROWS, int V, int R, int NW, int NST, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB) gated_bwd_kernel(const GatedArgs A) {
    using Lay = BwdLayout<XT, ZM, ROWS, V, R, NW, NST>;
    using ZT = typename Lay::ZT;
    constexpr int GATE = FORM / 3, WRITE = FORM % 3, L = NW * R, PAIR = Lay::PAIR, HO = Lay::HO, N = V / 2;
    constexpr bool HEAD = ZM == kZHead, VEC = ROWS != kAny;
    constexpr int NG = HEAD ? 1 : N;
    static_assert(R == kGatedMark, "a run starts at a mark");
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sw = reinterpret_cast<float*>(smem + Lay::SW) + lane * PAIR;
    float* sc = reinterpret_cast<float*>(smem + Lay::SC);
    const int K = A.K, rank = blockIdx.x % K;
    const int ct = (blockIdx.x / K) % A.ctiles, b = blockIdx.x / K / A.ctiles;
    const int c0 = ct * 32 * V, c = c0 + lane * V, n = A.C - c;
    const bool on = n > 0;
    const XT* x = static_cast<const XT*>(A.x) + (long long)b * A.xbs + c0;
    const XT* dy = static_cast<const XT*>(A.dy) + (long long)b * A.dybs + c0;
    const ZT* z = static_cast<const ZT*>(A.z) + (long long)b * A.zbs + c0;
    const int nz = HEAD ? A.C / A.d : A.C;  // gates per token
    XT* dx = static_cast<XT*>(A.dx) + (long long)b * A.T * A.C + c;
    const long long dzoff = (long long)b * A.T * nz + (HEAD ? c / A.d : c);
    const float* marks = A.marks + (long long)b * A.nmarks * A.C + c;
    const int len = row_length(A, b);
    const int iters = (len + K * L - 1) / (K * L);

    F2 g[N];  // a_{t+1} g_{t+1} of the first token behind the iteration (one CTA: the first warp's)
    load_state<VEC, N>(A.dh_T ? A.dh_T + (long long)b * A.C + c : nullptr, n, g);
    if (K == 1 && warp == 0) write_pairs<N>(sc + lane * V, g);

    Exchange ex(reinterpret_cast<uint64_t*>(smem + Lay::SB), reinterpret_cast<volatile uint32_t*>(smem + Lay::SB + 16),
                K * 32 * PAIR * 4, K > 1);
    unsigned char* mine = smem + warp * NST * Lay::STAGE;
    int ts = ((iters - 1) * K + rank) * L + warp * R;  // the run that is staged next
    Stager<ROWS, XT, V, R> sx(A.x, x, A.xts, A.C - c0, ts, -K * L, lane), sd(A.dy, dy, A.dyts, A.C - c0, ts, -K * L, lane);
    Stager<ROWS, ZT, V, R> sz(A.z, z, A.zts, A.C - c0, HEAD ? 0 : ts, -K * L, lane);
    const RowStart<ROWS, XT> x_at(x, A.xts), dy_at(dy, A.dyts);
    const RowStart<ROWS, ZT> z_at(z, A.zts);
    HeadGates<XT, V, R, 4> hg(A, b, c0, lane);
    auto stage = [&](int slot) {
        if (ts >= 0) {
            if (ts < len) {
                unsigned char* s = mine + slot * Lay::STAGE;
                sx.copy(reinterpret_cast<XT*>(s), len - ts, lane);
                sd.copy(reinterpret_cast<XT*>(s + Lay::X), len - ts, lane);
                if (on) {
                    const float* m = marks + (long long)(ts / kGatedMark) * A.C;
                    float* to = reinterpret_cast<float*>(s + Lay::M) + lane * V;
                    if constexpr (VEC) {
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                                     "l"(m), "n"(V * 4)
                                     : "memory");
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (v < n)
                                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to + v)),
                                             "l"(m + v)
                                             : "memory");
                    }
                }
                if constexpr (HEAD) hg.stage(A, reinterpret_cast<uint32_t*>(s + 2 * Lay::X), ts, len, lane);
                else sz.copy(reinterpret_cast<ZT*>(s + 2 * Lay::X), len - ts, lane);
            }
            sx.p += sx.move, sd.p += sd.move;
            if constexpr (!HEAD) sz.p += sz.move;
            ts -= K * L;
        }
        stage_commit();
    };
    float* gates = reinterpret_cast<float*>(smem + Lay::HG) + warp * (HeadGates<XT, V, R, 4>::BYTES / 4);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) stage(s);
    int slot = 0;
    for (int it = iters - 1; it >= 0; --it) {
        const int t0 = (it * K + rank) * L + warp * R, buf = (iters - 1 - it) & 1;
        stage(slot == 0 ? NST - 1 : slot - 1);
        stage_wait<NST - 1>();
        XT* xw = reinterpret_cast<XT*>(mine + slot * Lay::STAGE);
        XT* dw = reinterpret_cast<XT*>(mine + slot * Lay::STAGE + Lay::X);
        ZT* zw = reinterpret_cast<ZT*>(mine + slot * Lay::STAGE + 2 * Lay::X);
        slot = slot == NST - 1 ? 0 : slot + 1;
        const bool full = t0 + R <= len;
        if (!full) {
            fill_rows<XT, Lay::XROW, R>(xw, len - t0, 0.f, lane);
            fill_rows<XT, Lay::XROW, R>(dw, len - t0, 0.f, lane);
            if constexpr (!HEAD) fill_rows<ZT, Lay::ZROW, R>(zw, len - t0, neutral_z<GATE>(), lane);
            __syncwarp();
        }
        if constexpr (HEAD) {  // gate, write scale, its slope (unit write)
            hg.read(A, reinterpret_cast<const uint32_t*>(zw), t0, len, neutral_z<GATE>(), lane);
            hg.keep(gates, lane, [&](F2 hz, F2* out) {
                F2 hq;
                gates_of<GATE>(hz, A, false, out[0], hq);
                out[1] = writes_of<GATE, WRITE>(out[0], hq);
                out[2] = WRITE == kUnit ? unit_slopes(out[0], out[1]) : f2(0.f);
                out[3] = f2(0.f);
            });
        }
        uint32_t slow = ~0u;  // rows of which some gate needs more
        if constexpr (!HEAD && GATE == kLogitTau)
            if (A.squares == 0) slow = negative_rows<ROWS, ZT, N, R>(z_at, zw + lane * V, Lay::ZROW, t0);
        // Of each token: a, then the product of the run's gates behind it; s (per head it stays
        // in shared memory); dz / g, per head without da/dz; the run's own adjoint, from 0.
        F2 a[R][NG], s[HEAD ? 1 : R][NG], k[R][N], gl[R][N], h[N];
        read_pairs<float, N>(reinterpret_cast<const float*>(reinterpret_cast<unsigned char*>(xw) + Lay::M) + lane * V, h);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            F2 xf[N], zf[N], hs = f2(0.f);
            read_row<ROWS, XT, N>(x_at.row(xw + lane * V, Lay::XROW, t0, r), xf);
            if constexpr (HEAD) {
                F2 t[WRITE == kUnit ? 4 : 2];
                hg.template get<WRITE == kUnit ? 4 : 2>(gates, r, t);
                a[r][0] = t[0], s[0][0] = t[1];
                if constexpr (WRITE == kUnit) hs = t[2];
            } else {
                read_row<ROWS, ZT, N>(z_at.row(zw + lane * V, Lay::ZROW, t0, r), zf);
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int i = HEAD ? 0 : v;
                F2 q;
                if constexpr (!HEAD) {
                    gates_of<GATE>(zf[v], A, !(slow >> r & 1u), a[r][i], q);
                    s[r][i] = writes_of<GATE, WRITE>(a[r][i], q);
                    if constexpr (WRITE == kUnit) hs = unit_slopes(a[r][i], s[r][i]);
                }
                F2 m = h[v];  // d h_t / d a_t
                if constexpr (WRITE == kLeaky) m = fma2(xf[v], f2(-1.f), m);
                if constexpr (WRITE == kUnit) m = fma2(xf[v], hs, m);
                if constexpr (!HEAD && GATE != kValue) m = mul2(slopes_of<GATE>(zf[v], A.tau, a[r][i], q), m);
                k[r][v] = m;
                if (r < R - 1) h[v] = fma2(a[r][i], h[v], WRITE == kPlain ? xf[v] : mul2(s[HEAD ? 0 : r][i], xf[v]));
            }
        }
        F2 P[NG], G[N];
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            read_row<ROWS, XT, N>(dy_at.row(dw + lane * V, Lay::XROW, t0, r), gl[r]);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                if (r < R - 1) gl[r][v] = add2(gl[r][v], G[v]);
                G[v] = mul2(a[r][HEAD ? 0 : v], gl[r][v]);
            }
#pragma unroll
            for (int v = 0; v < NG; ++v) {
                const F2 t = a[r][v];
                a[r][v] = r < R - 1 ? P[v] : f2(1.f);
                P[v] = r < R - 1 ? mul2(P[v], t) : t;
            }
        }
        {
            float* p = sw + (buf * NW + warp) * 32 * PAIR;
            write_pairs<NG>(p, P);
            write_pairs<N>(p + HO, G);
        }
        __syncthreads();
        auto fold = [&](const float* p, const float* add, F2* state) {
            F2 p_[NG], h_[N];
            read_pairs<float, NG>(p, p_);
            read_pairs<float, N>(add, h_);
#pragma unroll
            for (int v = 0; v < N; ++v) state[v] = fma2(p_[HEAD ? 0 : v], state[v], h_[v]);
        };
        // the adjoint that enters it from behind
        F2 gin[N];
        if (K == 1) {
            read_pairs<float, N>(sc + (buf * 32 + lane) * V, gin);
        } else {
            if (warp < K) {
                F2 p_[NG], h_[N];
#pragma unroll
                for (int v = 0; v < NG; ++v) p_[v] = f2(1.f);
#pragma unroll
                for (int v = 0; v < N; ++v) h_[v] = f2(0.f);
#pragma unroll
                for (int w = NW - 1; w >= 0; --w) {
                    const float* p = sw + (buf * NW + w) * 32 * PAIR;
                    F2 t[NG];
                    fold(p, p + HO, h_);
                    read_pairs<float, NG>(p, t);
#pragma unroll
                    for (int v = 0; v < NG; ++v) p_[v] = mul2(p_[v], t[v]);
                }
                float f[PAIR] = {};
#pragma unroll
                for (int v = 0; v < NG; ++v) parts(p_[v], f[2 * v], f[2 * v + 1]);
#pragma unroll
                for (int v = 0; v < N; ++v) parts(h_[v], f[HO + 2 * v], f[HO + 2 * v + 1]);
                for (int k = warp; k < K; k += NW) ex.send<PAIR>(sc + ((buf * K + rank) * 32 + lane) * PAIR, k, buf, f);
            }
            ex.wait(buf, (iters - 1 - it) >> 1);
            for (int k = K - 1; k >= 0; --k) {
                if (k == rank) {
#pragma unroll
                    for (int v = 0; v < N; ++v) gin[v] = g[v];
                }
                const float* p = sc + ((buf * K + k) * 32 + lane) * PAIR;
                fold(p, p + HO, g);
            }
        }
        for (int w = NW - 1; w > warp; --w) {
            const float* p = sw + (buf * NW + w) * 32 * PAIR;
            fold(p, p + HO, gin);
        }
        if (K == 1 && warp == 0) {
#pragma unroll
            for (int v = 0; v < N; ++v) g[v] = fma2(P[HEAD ? 0 : v], gin[v], G[v]);
            write_pairs<N>(sc + ((buf ^ 1) * 32 + lane) * V, g);
        }
        // per head: the lanes' shares of dz, [R][36], where x and dy stood
        float* sums = reinterpret_cast<float*>(xw);
        static_assert(!HEAD || R * 36 * 4 <= 2 * Lay::X, "the stages hold the shares");
        if constexpr (HEAD) __syncwarp();
        XT* dxt = dx + (long long)t0 * A.C;
        ZT* dzt = static_cast<ZT*>(A.dz) + dzoff + (long long)t0 * nz;
        auto put = [&](int r, bool in) {
            F2 dxf[N], dzf[N], t[2];
            if constexpr (HEAD && WRITE != kPlain) hg.template get<2>(gates, r, t);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int i = HEAD ? 0 : v;
                const F2 g_ = r < R - 1 ? fma2(a[r][i], gin[v], gl[r][v]) : add2(gin[v], gl[r][v]);
                dxf[v] = WRITE == kPlain ? g_ : mul2(HEAD ? t[1] : s[HEAD ? 0 : r][i], g_);
                dzf[v] = mul2(k[r][v], g_);
            }
            if (in) store_row<VEC, XT, N>(dxt + (long long)r * A.C, dxf, n, lane);
            if constexpr (HEAD) {
                F2 sum = dzf[0];
#pragma unroll
                for (int v = 1; v < N; ++v) sum = add2(sum, dzf[v]);
                float lo, hi;
                parts(sum, lo, hi);
                sums[r * 36 + lane] = on ? lo + hi : 0.f;
            } else if (in) {
                store_row<VEC, ZT, N>(dzt + (long long)r * nz, dzf, n, lane);
            }
        };
        if (full && (on || !VEC)) {
#pragma unroll
            for (int r = 0; r < R; ++r) put(r, true);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) put(r, (on || !VEC) && t0 + r < len);
        }
        if constexpr (HEAD) {  // a head's d channels are those of d/V lanes; the gate's lane adds them up
            __syncwarp();
            hg.each_gate([&](int m, int r, int hd, F2 hz) {
                if (t0 + r >= len) return;
                const float* p = sums + r * 36 + hd * (A.d / V);
                float4 t = *reinterpret_cast<const float4*>(p);
                for (int i = 4; i < A.d / V; i += 4) {
                    const float4 u = *reinterpret_cast<const float4*>(p + i);
                    t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
                }
                float v = (t.x + t.y) + (t.z + t.w);
                if constexpr (GATE != kValue) {
                    F2 ga, gq;
                    gates_of<GATE>(hz, A, false, ga, gq);
                    float lo, hi;
                    parts(slopes_of<GATE>(hz, A.tau, ga, gq), lo, hi);
                    v *= m ? hi : lo;
                }
                const long long o = ((long long)b * A.T + t0 + r) * nz + c0 / A.d + hd;
                if (sizeof(XT) == 4 || A.z32) static_cast<float*>(A.dz)[o] = v;
                else static_cast<XT*>(A.dz)[o] = from_f<XT>(v);
            }, lane);
        }
        __syncwarp();  // the stage is read to its end before it is filled again
    }
    if (K > 1) cluster_sync_all();
    if (!on) return;
    if (rank == 0 && warp == 0) store_pairs<VEC, float, N>(A.dh0 + (long long)b * A.C + c, g, n);
    const float zero[V] = {};
    for (int t = len + rank * NW + warp; t < A.T; t += K * NW) {
        store_vec<VEC, XT, V>(dx + (long long)t * A.C, zero, n);
        const long long o = dzoff + (long long)t * nz;
        if constexpr (HEAD) {
            if (lane % (A.d / V) == 0) {
                if (sizeof(XT) == 4 || A.z32) static_cast<float*>(A.dz)[o] = 0.f;
                else static_cast<XT*>(A.dz)[o] = from_f<XT>(0.f);
            }
        } else {
            store_vec<VEC, ZT, V>(static_cast<ZT*>(A.dz) + o, zero, n);
        }
    }
}

// ---- one token: h_out = a h + s(a) x, y = h_out. One thread per V channels.
template <class XT, int ZM, int FORM, bool VEC, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedArgs A) {
    using ZT = typename std::conditional<ZM == kZ32, float, XT>::type;
    constexpr int GATE = FORM / 3, WRITE = FORM % 3;
    const int vecs = (A.C + V - 1) / V;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)vecs * A.B) return;
    const int b = (int)(i / vecs), c = (int)(i % vecs) * V, n = A.C - c;
    const long long o = (long long)b * A.C + c;
    const Vec<XT, V> xr = load_vec<VEC, XT, V>(static_cast<const XT*>(A.x) + (long long)b * A.xbs + c, n);
    float zf[V];
    if constexpr (ZM == kZHead) {
        const float zh = load_gate<XT>(A.z, (long long)b * A.zbs + c / A.d, A.z32);
#pragma unroll
        for (int v = 0; v < V; ++v) zf[v] = zh;
    } else {
        const Vec<ZT, V> zr = load_vec<VEC, ZT, V>(static_cast<const ZT*>(A.z) + (long long)b * A.zbs + c, n);
#pragma unroll
        for (int v = 0; v < V; ++v) zf[v] = to_f(zr.v[v]);
    }
    Vec<float, V> h = load_vec<VEC, float, V>(A.h0 + o, n);
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        F2 a, q;
        gates_of<GATE>(f2(zf[v], zf[v + 1]), A, false, a, q);
        const F2 u = mul2(writes_of<GATE, WRITE>(a, q), f2(to_f(xr.v[v]), to_f(xr.v[v + 1])));
        parts(fma2(a, f2(h.v[v], h.v[v + 1]), u), h.v[v], h.v[v + 1]);
    }
    store_vec<VEC, float, V>(A.h_out + o, h.v, n);
    store_vec<VEC, XT, V>(static_cast<XT*>(A.y) + o, h.v, n);
}

}  // namespace gated
}  // namespace lattice

// selective_bwd.cuh -- backward pass of the selective scan (formulas and layout: selective.cuh).
//
// A CTA takes its segment's tiles of 16 tokens from the last to the first. The forward pass left the state
// before every kSelMark-th token; from it a thread recomputes 8 tokens' states, keeps them and their decays in
// registers, and goes back through them with the cotangent g.
//
// Sums over a channel's states (y, du, and ddt's part) are shuffles over its L lanes as in the forward pass. Sums
// over channels (db, dc) are shuffles over the warp's channels; a lane names its four states so that what it
// keeps and what it hands on have the same registers in all lanes (register r stands for state r ^ (channel & 3)),
// which takes the selects out of the first two steps; shared memory adds the warps up, the workspace the CTAs. All in a
// fixed order.
#pragma once
#include "selective.cuh"

namespace lattice {
namespace selective {

template <class XT, int L>
struct BwdShared {
    static constexpr int NP = 4 * L, CT = Place<L>::CT, CTP = Place<L>::CTP;
    static constexpr int VAR = L <= 8 ? 4 : L == 16 ? 2 : 1;  // orders of a lane's four states
    static constexpr int VS = TT * NP + (NP < 32 ? NP : 0);   // from order to order, apart in the banks
    ulonglong2 dtu[TT * CT];                                  // (dt, dt, u, u), u = dt x
    F2 w[TT * CT];                                            // (w, w)
    F2 x[TT * CT / 2], slope[TT * CT / 2], zf[TT * CT / 2];   // of pairs of channels, for the thread that wrote them
    float y[TT * CTP], du[TT * CTP], dq[TT * CTP];            // sums over n
    float b[VAR * VS], c[VAR * VS];
    float sums[2][NW][TT * NP];                               // dc and db of the warps' channels
};

// the lane's states from register order to memory order, and back
template <int VAR>
__device__ __forceinline__ void reorder(float* v, int order) {
    if constexpr (VAR >= 2) {
        const bool o = order & 1;
        const float a = o ? v[1] : v[0], b = o ? v[0] : v[1], c = o ? v[3] : v[2], d = o ? v[2] : v[3];
        v[0] = a, v[1] = b, v[2] = c, v[3] = d;
    }
    if constexpr (VAR >= 4) {
        const bool o = order & 2;
        const float a = o ? v[2] : v[0], b = o ? v[3] : v[1], c = o ? v[0] : v[2], d = o ? v[1] : v[3];
        v[0] = a, v[1] = b, v[2] = c, v[3] = d;
    }
}
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Sums over the warp's channels of four states, token by token from the last: what add() has taken is written by the call
// for which it has enough tokens.
template <int L>
struct ChannelSums {
    static constexpr int NP = 4 * L;
    float v1, r23, v3;
    __device__ __forceinline__ void add(float* out, int t, const F2* f, int lane, int gl, int cl) {
        float s[4];
        parts(f[0], s[0], s[1]), parts(f[1], s[2], s[3]);
        if constexpr (L <= 8) {
            s[0] += __shfl_xor_sync(ALL, s[2], 2 * L);
            s[1] += __shfl_xor_sync(ALL, s[3], 2 * L);
            s[0] += __shfl_xor_sync(ALL, s[1], L);
            const int at = gl * 4 + (cl & 3);
            if constexpr (L == 8) {
                out[t * NP + at] = s[0];
            } else if constexpr (L == 4) {
                if (t & 1) v1 = s[0];
                else out[(t + (lane >> 4)) * NP + at] = halve(s[0], v1, lane, 16);
            } else {
                if ((t & 3) == 3) v3 = s[0];
                else if ((t & 3) == 2) r23 = halve(s[0], v3, lane, 8);
                else if ((t & 3) == 1) v1 = s[0];
                else out[(t + (lane >> 3)) * NP + at] = halve(halve(s[0], v1, lane, 8), r23, lane, 16);
            }
        } else if constexpr (L == 16) {
            s[0] += __shfl_xor_sync(ALL, s[1], 16);
            s[2] += __shfl_xor_sync(ALL, s[3], 16);
            out[t * NP + gl * 4 + cl] = s[0];
            out[t * NP + gl * 4 + (2 ^ cl)] = s[2];
        } else {
            *reinterpret_cast<float4*>(out + t * NP + gl * 4) = make_float4(s[0], s[1], s[2], s[3]);
        }
    }
};
// Sums over a channel's lanes of one value, four tokens at a time from the last; out: [TT][CTP].
template <int L>
struct StateSums {
    float v1, v3, r23;
    __device__ __forceinline__ void add(float* out, int stride, int t, float s, int lane, int gl, int c) {
        if ((t & 3) == 3) {
            v3 = s;
        } else if ((t & 3) == 2) {
            r23 = halve(s, v3, lane, 1);
        } else if ((t & 3) == 1) {
            v1 = s;
        } else {
            const float r01 = halve(s, v1, lane, 1);
            if constexpr (L == 2) {
                out[(t + gl) * stride + c] = r01;
                out[(t + 2 + gl) * stride + c] = r23;
            } else {
                float v = halve(r01, r23, lane, 2);
#pragma unroll
                for (int o = 4; o < L; o *= 2) v += __shfl_xor_sync(ALL, v, o);
                if (gl < 4) out[(t + gl) * stride + c] = v;
            }
        }
    }
};

template <class XT, int L, bool GATE>
__global__ void __launch_bounds__(NT, L == 32 ? 1 : 2) bwd_kernel(const SelArgs A) {
    using P = Place<L>;
    using Sh = BwdShared<XT, L>;
    constexpr int NP = Sh::NP, CT = P::CT, CTP = P::CTP, PI = P::PI, NB = Rows<NP>::NB, VAR = Sh::VAR, VS = Sh::VS, SB = 8;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh& sh = *reinterpret_cast<Sh*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * 4, pw = p.width(), order = p.cl & (VAR - 1), warp = threadIdx.x >> 5;
    const long long EN = (long long)A.E * A.N, own = (long long)p.ch * A.N, seg = (long long)p.b * A.nseg + p.s;
    F2 g[2], A2[2], dA[2] = {f2(0.f), f2(0.f)}, bias = f2(0.f), skip = f2(0.f), dskip = f2(0.f), dbias = f2(0.f);
    {
        float v[4] = {};
        if (p.live) load_states<4>(A.A + own, n0, A.N, A.vec_n, v);
        reorder<VAR>(v, order);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= kLog2e;
        pack<4>(v, A2);
        const float* from = A.nseg > 1 ? A.seg_state + seg * EN : A.dh_T ? A.dh_T + p.b * EN : nullptr;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = 0.f;
        if (from && p.live) load_states<4>(from + own, n0, A.N, A.vec_n, v);
        reorder<VAR>(v, order);
        pack<4>(v, g);
        if (A.dt_bias) bias = value2(load2<float>(A.dt_bias, p.pair(), pw, false));
        if (A.skip) skip = value2(load2<float>(A.skip, p.pair(), pw, false));
    }
    const long long xat = p.b * A.xbs + p.pair(), dat = p.b * A.dbs + p.pair(), zat = p.b * A.zbs + p.pair(),
                    yat = p.b * A.ybs + p.pair(), bat = p.b * A.bbs + p.g * A.N, cat = p.b * A.cbs + p.g * A.N,
                    oat = (long long)p.b * A.T * A.E + p.pair();
    const float* marks = A.marks + (long long)p.b * A.nmarks * EN + own;
    auto put_dt = [&](long long i, F2 v, int n) {
        if (sizeof(XT) == 4 || A.dt32) store2<float>(A.ddt, i, v, n, A.vec);
        else store2<XT>(A.ddt, i, v, n, A.vec);
    };
    auto mark = [&](int t, F2* h) {  // the state before token t
        float v[4] = {};
        if (p.live && t < p.te) load_states<4>(marks + (long long)(t / kSelMark) * EN, n0, A.N, A.vec_n, v);
        reorder<VAR>(v, order);
        pack<4>(v, h);
    };
    auto stage = [&](int tb) {
        Pair<XT> rx[PI], rz[PI] = {}, ry[PI];
        Pair<float> rd[PI];
        XT rb[NB], rc[NB];
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load2<XT>(A.x, xat + t * A.xts, n, A.vec);
            rd[k] = load_dt<XT>(A, dat + t * A.dts, n);
            ry[k] = load2<XT>(A.dy, yat + t * A.yts, n, A.vec);
            if constexpr (GATE) rz[k] = load2<XT>(A.z, zat + t * A.zts, n, A.vec);
        }
        fetch_rows<XT, NP>(A.b, bat, A.bts, tb, p.te, A.N, rb);
        fetch_rows<XT, NP>(A.c, cat, A.cts, tb, p.te, A.N, rc);
        if (tb > p.t0) {  // the next tile's lines are brought nearer
#pragma unroll
            for (int k = 0; k < PI; ++k) {
                const int r = p.row + k * P::ROWS, t = tb - TT + r;
                if (r >= TT || pw == 0) continue;
                const char *px = static_cast<const char*>(A.x) + (xat + t * A.xts) * (long long)sizeof(XT),
                           *py = static_cast<const char*>(A.dy) + (yat + t * A.yts) * (long long)sizeof(XT),
                           *pd = static_cast<const char*>(A.dt) + (dat + t * A.dts) * (long long)(A.dt32 ? 4 : sizeof(XT));
                prefetch(px), prefetch(py), prefetch(pd);
                if constexpr (GATE) prefetch(static_cast<const char*>(A.z) + (zat + t * A.zts) * (long long)sizeof(XT));
            }
            if (p.live && n0 < A.N)
#pragma unroll
                for (int t = 0; t < TT; t += kSelMark) prefetch(marks + (long long)((tb - TT + t) / kSelMark) * EN + n0);
        }
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (r >= TT) continue;
            F2 dt = f2(0.f), u = f2(0.f), w = f2(0.f), slope = f2(0.f), zf = f2(0.f), x = f2(0.f);
            if (tb + r < p.te) {
                dt = step_size<XT>(A, rd[k], bias, &slope);
                x = value2(rx[k]);
                u = mul2(dt, x);
                w = value2(ry[k]);
                if constexpr (GATE) {  // dy silu(z), dy silu'(z)
                    const F2 z = value2(rz[k]), s = sigmoid(z), zs = mul2(z, s);
                    zf = mul2(w, fma2(zs, fma2(s, f2(-1.f), f2(1.f)), s));
                    w = mul2(w, zs);
                }
            }
            float d0, d1, u0, u1, w0, w1;
            parts(dt, d0, d1), parts(u, u0, u1), parts(w, w0, w1);
            const int at = r * CT + 2 * p.cp;
            sh.dtu[at] = both(f2(d0), f2(u0));
            sh.dtu[at + 1] = both(f2(d1), f2(u1));
            *reinterpret_cast<ulonglong2*>(sh.w + at) = both(f2(w0), f2(w1));
            sh.x[at / 2] = x, sh.slope[at / 2] = slope;
            if constexpr (GATE) sh.zf[at / 2] = zf;
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i >= TT * NP) continue;
            const float vb = to_f(rb[k]), vc = to_f(rc[k]);
#pragma unroll
            for (int v = 0; v < VAR; ++v) sh.b[v * VS + (i ^ v)] = vb, sh.c[v * VS + (i ^ v)] = vc;
        }
    };
    auto finish = [&](int tb) {  // the tile's outputs
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r;
            if (r >= TT || t >= p.te) continue;
            const int at = r * CT + 2 * p.cp, st = r * CTP + 2 * p.cp;
            const ulonglong2 p0 = sh.dtu[at], p1 = sh.dtu[at + 1], ww = *reinterpret_cast<const ulonglong2*>(sh.w + at);
            float d0, d1, w0, w1, other;
            parts(low(p0), d0, other), parts(low(p1), d1, other), parts(F2{ww.x}, w0, other), parts(F2{ww.y}, w1, other);
            const F2 x = sh.x[at / 2], w = f2(w0, w1), du = *reinterpret_cast<const F2*>(sh.du + st);
            const long long o = oat + (long long)t * A.E;
            store2<XT>(A.dx, o, fma2(du, f2(d0, d1), mul2(skip, w)), pw, A.vec);
            const F2 ddt = mul2(fma2(*reinterpret_cast<const F2*>(sh.dq + st), f2(kLn2), mul2(du, x)), sh.slope[at / 2]);
            put_dt(o, ddt, pw);
            dbias = add2(dbias, ddt);
            dskip = fma2(w, x, dskip);
            if constexpr (GATE)
                store2<XT>(A.dz, o, mul2(fma2(skip, x, *reinterpret_cast<const F2*>(sh.y + st)), sh.zf[at / 2]), pw, A.vec);
        }
        float* out = A.parts_bc + (((long long)p.ct * A.B + p.b) * A.T + tb) * 2 * A.N;
        for (int i = threadIdx.x; i < 2 * TT * NP; i += NT) {
            const int kind = i / (TT * NP), j = i - kind * TT * NP, t = j / NP, n = j % NP;
            if (n >= A.N || tb + t >= p.te) continue;
            float v = sh.sums[kind][0][j];
#pragma unroll
            for (int q = 1; q < NW; ++q) v += sh.sums[kind][q][j];
            out[(long long)t * 2 * A.N + kind * A.N + n] = v;
        }
    };
    const int tiles = (p.te - p.t0 + TT - 1) / TT;
    for (int i = tiles - 1; i >= 0; --i) {
        const int tb = p.t0 + i * TT;
        __syncthreads();
        if (i + 1 < tiles) finish(tb + TT);
        stage(tb);
        __syncthreads();
        F2 sA[2] = {f2(0.f), f2(0.f)};
        StateSums<L> sy, sd, sq;
        ChannelSums<L> sb, sc;
        const float *vb = sh.b + order * VS + n0, *vc = sh.c + order * VS + n0;
#pragma unroll 1
        for (int q = TT - SB; q >= 0; q -= SB) {
            F2 a[SB][2], hp[SB][2], h[2];
            mark(tb + q / kSelMark * kSelMark, h);
            if (kSelMark > SB && q) {
#pragma unroll
                for (int t = 0; t < SB; ++t) {
                    const ulonglong2 du = sh.dtu[t * CT + p.c];
                    F2 bv[2];
                    read_vec<4>(vb + t * NP, bv);
#pragma unroll
                    for (int k = 0; k < 2; ++k) h[k] = fma2(decay(mul2(low(du), A2[k])), h[k], mul2(high(du), bv[k]));
                }
            }
#pragma unroll
            for (int j = 0; j < SB; ++j) {
                const ulonglong2 du = sh.dtu[(q + j) * CT + p.c];
                F2 bv[2];
                read_vec<4>(vb + (q + j) * NP, bv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    hp[j][k] = h[k];
                    a[j][k] = decay(mul2(low(du), A2[k]));
                    h[k] = fma2(a[j][k], h[k], mul2(high(du), bv[k]));
                }
            }
#pragma unroll
            for (int j = SB - 1; j >= 0; --j) {
                const int t = q + j;
                const ulonglong2 du = sh.dtu[t * CT + p.c];
                const F2 w = sh.w[t * CT + p.c];
                F2 bv[2], cv[2], dc[2], db[2], yy, dd, qq;
                read_vec<4>(vb + t * NP, bv);
                read_vec<4>(vc + t * NP, cv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    dc[k] = mul2(w, h[k]);
                    if constexpr (GATE) yy = k ? fma2(h[k], cv[k], yy) : mul2(h[k], cv[k]);
                    g[k] = fma2(w, cv[k], g[k]);
                    db[k] = mul2(high(du), g[k]);
                    dd = k ? fma2(g[k], bv[k], dd) : mul2(g[k], bv[k]);
                    g[k] = mul2(a[j][k], g[k]);
                    const F2 ah = mul2(g[k], hp[j][k]);
                    qq = k ? fma2(ah, A2[k], qq) : mul2(ah, A2[k]);
                    sA[k] = fma2(ah, low(du), sA[k]);
                    h[k] = hp[j][k];
                }
                // j stands for t in the choice of what is handed on: q is a multiple of 4
                if constexpr (GATE) sy.add(sh.y + q * CTP, CTP, j, total(yy), p.lane, p.gl, p.c);
                sd.add(sh.du + q * CTP, CTP, j, total(dd), p.lane, p.gl, p.c);
                sq.add(sh.dq + q * CTP, CTP, j, total(qq), p.lane, p.gl, p.c);
                sc.add(sh.sums[0][warp] + q * NP, j, dc, p.lane, p.gl, p.cl);
                sb.add(sh.sums[1][warp] + q * NP, j, db, p.lane, p.gl, p.cl);
            }
        }
        dA[0] = add2(dA[0], sA[0]), dA[1] = add2(dA[1], sA[1]);  // tile by tile: short sums lose less
    }
    __syncthreads();
    if (tiles) finish(p.t0);
    for (int t = p.te + p.row; t < p.t1; t += P::ROWS) {  // behind the sequence's end
        const long long o = oat + (long long)t * A.E;
        store2<XT>(A.dx, o, f2(0.f), pw, A.vec);
        put_dt(o, f2(0.f), pw);
        if constexpr (GATE) store2<XT>(A.dz, o, f2(0.f), pw, A.vec);
    }
    if (p.live) {
        float v[4];
        unpack<4>(dA, v);
        reorder<VAR>(v, order);
        store_states<4>(A.parts_A + seg * EN + own, n0, A.N, A.vec_n, v);
        if (p.s == 0) {
            unpack<4>(g, v);
            reorder<VAR>(v, order);
            store_states<4>(A.dh0 + p.b * EN + own, n0, A.N, A.vec_n, v);
        }
    }
    // the sums over tokens per channel: row by row, in order
    __syncthreads();
    float4* rows = reinterpret_cast<float4*>(raw_shared);
    float s0, s1, k0, k1;
    parts(dskip, s0, s1), parts(dbias, k0, k1);
    rows[threadIdx.x] = make_float4(s0, s1, k0, k1);
    __syncthreads();
    if (p.row == 0) {
        for (int r = 1; r < P::ROWS; ++r) {
            const float4 o = rows[r * P::PAIRS + p.cp];
            s0 += o.x, s1 += o.y, k0 += o.z, k1 += o.w;
        }
        float* out = A.parts_ch + seg * 2 * A.E + p.pair();
        if (pw > 0) out[0] = s0, out[A.E] = k0;
        if (pw > 1) out[1] = s1, out[A.E + 1] = k1;
    }
}

// db and dc from the channel tiles' sums, in their order
template <class XT>
__global__ void __launch_bounds__(256) shared_kernel(const SelArgs A) {
    const int n2 = 2 * A.N;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, rows = (long long)A.B * A.T;
    if (i >= rows * A.G * n2) return;
    const long long r = i / n2, bt = r / A.G;
    const int m = (int)(i - r * n2), g = (int)(r - bt * A.G), b = (int)(bt / A.T), kind = m >= A.N, n = m - kind * A.N;
    const int len = A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
    float v = 0.f;
    if (bt - (long long)b * A.T < len) {
        const float* from = A.parts_bc + ((long long)g * A.tiles * rows + bt) * n2 + m;
#pragma unroll 8
        for (int k = 0; k < A.tiles; ++k) v += from[k * rows * n2];
    }
    put(static_cast<XT*>(kind ? A.db : A.dc) + r * A.N + n, v);
}

// dA, dskip and ddt_bias from the segments' sums, in their order
inline __global__ void __launch_bounds__(256) weights_kernel(const SelArgs A) {
    const long long EN = (long long)A.E * A.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= EN + 2 * A.E) return;
    const bool ch = i >= EN;
    const float* from = ch ? A.parts_ch + (i - EN) : A.parts_A + i;
    const long long step = ch ? 2 * A.E : EN;
    float v = 0.f;
#pragma unroll 4
    for (int k = 0; k < A.B * A.nseg; ++k) v += from[k * step];
    if (!ch) A.dA[i] = v;
    else if (i - EN < A.E) {
        if (A.dskip) A.dskip[i - EN] = v;
    } else if (A.ddt_bias) {
        A.ddt_bias[i - EN - A.E] = v;
    }
}

}  // namespace selective
}  // namespace lattice

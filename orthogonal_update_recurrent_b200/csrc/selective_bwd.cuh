// selective_bwd.cuh -- backward pass of the selective scan (formulas and layout: selective.cuh).
//
// A CTA takes its segment's tiles of 16 tokens from the last to the first. The forward pass left the state
// before every kSelMark-th token; from it a thread recomputes 8 tokens' states, keeps them and their decays in
// registers, and goes back through them with the cotangent g.
//
// Sums over a channel's states (y, du) are taken as in the forward pass or, where the lanes' parts would take too much shared memory,
// by shuffles, four tokens at once (each lane hands half of its tokens on per step), and ddt's part always. Sums
// over channels (db, dc) are shuffles over the warp's channels; a lane names its four states so that what it
// keeps and what it hands on have the same registers in all lanes (register r stands for state r ^ (channel & 3)),
// which takes the selects out of the first two steps; shared memory adds the warps up, the workspace the CTAs. All in a
// fixed order.
//
// Mid-size layer (8 x 4096 tokens of 2048 bf16 channels, 16 states, gate): 1575 us, of which HBM would need 225, and 48 us for the sums
// over the channel tiles. A token costs a warp 116 instructions for 128 states: 58 % of the issue slots; shared memory and shuffles keep
// their pipe busy 65 % of the time, at 16 warps per SM (127 registers: 8 tokens' states and decays).
#pragma once
#include "selective.cuh"

namespace lattice {
namespace selective {

template <class XT, int L, int W>
struct BwdShared {
    static constexpr int NP = 4 * L, CT = Place<L, W>::CT, CTP = Place<L, W>::CTP;
    static constexpr int VAR = L <= 8 ? 4 : L == 16 ? 2 : 1;  // orders of a lane's four states
    static constexpr int VS = TT * NP + (NP < 32 ? NP : 0);   // from order to order, apart in the banks
    // The lanes' sums over n stand side by side for few lanes, whole for many: floats of a token
    static constexpr bool PARTS = L == 4 || L == 8;  // (two lanes' parts would leave one CTA per SM)
    static constexpr int WHOLE = CT + 8, ROW = PARTS ? L * CTP : WHOLE;
    float2 du[TT * Place<L, W>::DW];                             // (dt, u), u = dt x
    float w[TT * Place<L, W>::DW];
    float x[TT * CT], slope[TT * CT], zf[TT * CT];            // for the thread that wrote them
    float y[TT * ROW], g[TT * ROW], q[TT * WHOLE];            // the sums over n of y, du and (always whole) ddt's part
    float b[VAR * VS], c[VAR * VS];
    float sums[2][W][TT * NP];                               // dc and db of the warps' channels
    // for the threads' channels, what is added up over the tiles too: in registers they would cost spills
    float bias[CT], skip[CT], dskip[32 * W * Place<L, W>::V], dbias[32 * W * Place<L, W>::V];
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

// Sums over the warp's channels of four states of dc and of db, token by token from the last: what add() has taken is written by
// the call for which it has enough tokens. The two are added in pairs.
template <int L>
struct ChannelSums {
    static constexpr int NP = 4 * L;
    F2 v1, r23, v3;  // (dc, db)
    static __device__ __forceinline__ F2 shfl(F2 v, int o) {
        float a, b;
        parts(v, a, b);
        return f2(__shfl_xor_sync(ALL, a, o), __shfl_xor_sync(ALL, b, o));
    }
    static __device__ __forceinline__ F2 half(F2 v0, F2 v1, int lane, int bit) {  // halve() of both
        float a0, b0, a1, b1;
        parts(v0, a0, b0), parts(v1, a1, b1);
        const bool up = lane & bit;
        return add2(f2(up ? a1 : a0, up ? b1 : b0), shfl(f2(up ? a0 : a1, up ? b0 : b1), bit));
    }
    static __device__ __forceinline__ void put(float* dc, float* db, int at, F2 v) { parts(v, dc[at], db[at]); }
    __device__ __forceinline__ void add(float* dc, float* db, int t, const F2* c, const F2* b, int lane, int gl, int cl) {
        float c0, c1, b0, b1;
        if constexpr (L <= 8) {
            const F2 cs = add2(c[0], shfl(c[1], 2 * L)), bs = add2(b[0], shfl(b[1], 2 * L));
            parts(cs, c0, c1), parts(bs, b0, b1);
            const F2 s = add2(f2(c0, b0), shfl(f2(c1, b1), L));
            const int at = gl * 4 + (cl & 3);
            if constexpr (L == 8) {
                put(dc, db, t * NP + at, s);
            } else if constexpr (L == 4) {
                if (t & 1) v1 = s;
                else put(dc, db, (t + (lane >> 4)) * NP + at, half(s, v1, lane, 16));
            } else {
                if ((t & 3) == 3) v3 = s;
                else if ((t & 3) == 2) r23 = half(s, v3, lane, 8);
                else if ((t & 3) == 1) v1 = s;
                else put(dc, db, (t + (lane >> 3)) * NP + at, half(half(s, v1, lane, 8), r23, lane, 16));
            }
        } else if constexpr (L == 16) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                parts(c[k], c0, c1), parts(b[k], b0, b1);
                put(dc, db, t * NP + gl * 4 + (2 * k ^ cl), add2(f2(c0, b0), shfl(f2(c1, b1), 16)));
            }
        } else {
            *reinterpret_cast<ulonglong2*>(dc + t * NP + gl * 4) = make_ulonglong2(c[0].v, c[1].v);
            *reinterpret_cast<ulonglong2*>(db + t * NP + gl * 4) = make_ulonglong2(b[0].v, b[1].v);
        }
    }
};
// Sums over a channel's lanes of one value, four tokens at a time from the last; out: [.][stride]
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
            float v = halve(s, v1, lane, 1);
            if constexpr (L == 2) {
                out[(t + gl) * stride + c] = v;
                out[(t + 2 + gl) * stride + c] = r23;
            } else {
                v = halve(v, r23, lane, 2);
#pragma unroll
                for (int o = 4; o < L; o *= 2) v += __shfl_xor_sync(ALL, v, o);
                if (gl < 4) out[(t + gl) * stride + c] = v;
            }
        }
    }
};

template <class XT, int L, int W, bool GATE, bool VEC>
__global__ void __launch_bounds__(32 * W, L == 32 && W == 8 ? 1 : 16 / W) bwd_kernel(const SelArgs A) {
    using P = Place<L, W>;
    using Sh = BwdShared<XT, L, W>;
    constexpr int NT = P::NT, NP = Sh::NP, CT = P::CT, CTP = P::CTP, PI = P::PI, NB = Rows<NP, W>::NB, VAR = Sh::VAR, VS = Sh::VS, ROW = Sh::ROW, WHOLE = Sh::WHOLE, SB = kSelMark,
                  V = P::V, Q = P::P, DW = P::DW;
    static_assert(SB % 4 == 0 && TT % SB == 0, "tokens between marks: whole groups of the sums, whole parts of a tile");
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh& sh = *reinterpret_cast<Sh*>(raw_shared);
    const P p(A);
    const int n0 = p.gl * 4, pw = p.width(), order = p.cl & (VAR - 1), warp = threadIdx.x >> 5, entry = P::entry(p.c);
    const long long EN = (long long)A.E * A.N, own = (long long)p.ch * A.N, seg = (long long)p.b * A.nseg + p.s;
    F2 g[2], A2[2], dA[2] = {f2(0.f), f2(0.f)};
    {
        float v[4] = {};
        if (p.live) load_states<4>(A.A + own, n0, A.N, A.vec_n, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= kLog2e;
        float e[4];
        entering<L, W, 4, true>(A, p, n0, v, e);
        reorder<VAR>(v, order);
        pack<4>(v, A2);
        reorder<VAR>(e, order);
        pack<4>(e, g);
        F2 f[Q];
        load_columns<V>(A.dt_bias, p.column(), pw, f);
        if (p.row == 0) own_write<V>(sh.bias + p.first, f);
        load_columns<V>(A.skip, p.column(), pw, f);
        if (p.row == 0) own_write<V>(sh.skip + p.first, f);
#pragma unroll
        for (int q = 0; q < Q; ++q) f[q] = f2(0.f);
        own_write<V>(sh.dskip + threadIdx.x * V, f);
        own_write<V>(sh.dbias + threadIdx.x * V, f);
    }
    const XT *xp = static_cast<const XT*>(A.x) + p.b * A.xbs, *zp = static_cast<const XT*>(A.z) + p.b * A.zbs,
             *gp = static_cast<const XT*>(A.dy) + p.b * A.ybs, *bp = static_cast<const XT*>(A.b) + p.b * A.bbs + (long long)p.g * A.N,
             *cp = static_cast<const XT*>(A.c) + p.b * A.cbs + (long long)p.g * A.N;
    const void* dp = dt_at<XT>(A, p.b);
    const long long oat = (long long)p.b * A.T * A.E;
    const float* marks = A.marks + (long long)p.b * A.nmarks * EN + own;
    auto put_dt = [&](int t, const F2* v) {
        if (sizeof(XT) == 4 || A.dt32) store<VEC, float, V>(token<VEC>(static_cast<float*>(A.ddt) + oat, p.column(), t, A.E), v, pw);
        else store<VEC, XT, V>(token<VEC>(static_cast<XT*>(A.ddt) + oat, p.column(), t, A.E), v, pw);
    };
    auto put_x = [&](void* to, int t, const F2* v) { store<VEC, XT, V>(token<VEC>(static_cast<XT*>(to) + oat, p.column(), t, A.E), v, pw); };
    auto mark = [&](int t, F2* h) {  // the state before token t
        float v[4] = {};
        if (p.live && t < p.te) load_states<4>(marks + (long long)(t / kSelMark) * EN, n0, A.N, A.vec_n, v);
        reorder<VAR>(v, order);
        pack<4>(v, h);
    };
    Raw<XT, V> rx[PI], rz[PI], ry[PI];
    Raw<float, V> rd[PI];
    XT rb[NB], rc[NB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r, n = r < TT && t < p.te ? pw : 0;
            rx[k] = load<VEC, XT, V>(token<VEC>(xp, p.column(), t, A.xts), n);
            rd[k] = load_dt<VEC, XT, V>(A, dp, p.column(), t, n);
            ry[k] = load<VEC, XT, V>(token<VEC>(gp, p.column(), t, A.yts), n);
            if constexpr (GATE) rz[k] = load<VEC, XT, V>(token<VEC>(zp, p.column(), t, A.zts), n);
        }
        fetch_rows<VEC, XT, NP, W>(bp, A.bts, tb, p.te, A.N, rb);
        fetch_rows<VEC, XT, NP, W>(cp, A.cts, tb, p.te, A.N, rc);
    };
    auto ahead = [&](int tb) {  // a tile's lines are brought nearer
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r;
            if (r >= TT || pw == 0) continue;
            prefetch(token<VEC>(xp, p.column(), t, A.xts));
            prefetch(token<VEC>(gp, p.column(), t, A.yts));
            prefetch(sizeof(XT) == 4 || A.dt32 ? static_cast<const void*>(token<VEC>(static_cast<const float*>(dp), p.column(), t, A.dts))
                                               : static_cast<const void*>(token<VEC>(static_cast<const XT*>(dp), p.column(), t, A.dts)));
            if constexpr (GATE) prefetch(token<VEC>(zp, p.column(), t, A.zts));
        }
        if (p.live && n0 < A.N)
#pragma unroll
            for (int t = 0; t < TT; t += kSelMark) prefetch(marks + (long long)((tb + t) / kSelMark) * EN + n0);
    };
    auto prepare = [&](int tb) {
        F2 bias[Q], dskip[Q];
        own_read<V>(sh.bias + p.first, bias);
        own_read<V>(sh.dskip + threadIdx.x * V, dskip);
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS;
            if (TT % P::ROWS != 0 && r >= TT) continue;
            F2 dt[Q], slope[Q], x[Q], u[Q], w[Q], z[Q];
            step_sizes<XT, V>(A, rd[k], bias, dt, slope);
            values<XT, V>(rx[k], x);
            values<XT, V>(ry[k], w);
            if constexpr (GATE) values<XT, V>(rz[k], z);
            const bool in = tb + r < p.te;
            const int at = r * CT + p.first;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!in) dt[q] = f2(0.f);
                u[q] = mul2(dt[q], x[q]);  // rows behind the end were read as 0
                if constexpr (GATE) {      // dy silu(z), dy silu'(z)
                    const F2 s = sigmoid(z[q]), zs = mul2(z[q], s);
                    z[q] = mul2(w[q], fma2(zs, fma2(s, f2(-1.f), f2(1.f)), s));
                    w[q] = mul2(w[q], zs);
                }
                dskip[q] = fma2(w[q], x[q], dskip[q]);
            }
            p.write(sh.du, r, dt, u);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float w0, w1;
                parts(w[v / 2], w0, w1);
                sh.w[r * DW + P::entry(p.first + v)] = v & 1 ? w1 : w0;
            }
            own_write<V>(sh.x + at, x);
            own_write<V>(sh.slope + at, slope);
            if constexpr (GATE) own_write<V>(sh.zf + at, z);
        }
        own_write<V>(sh.dskip + threadIdx.x * V, dskip);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i >= TT * NP) continue;
            const float vb = to_f(rb[k]), vc = to_f(rc[k]);
#pragma unroll
            for (int v = 0; v < VAR; ++v) sh.b[v * VS + (i ^ v)] = vb, sh.c[v * VS + (i ^ v)] = vc;
        }
    };
    auto whole = [&](const float* rows, int r, F2* f) {  // the thread's channels' sums over n
        if constexpr (Sh::PARTS) lane_sums<L, W>(rows + r * ROW + p.first, f);
        else own_read<V>(rows + r * ROW + p.first, f);
    };
    auto finish = [&](int tb) {  // the tile's outputs
        F2 skip[Q], dbias[Q];
        own_read<V>(sh.skip + p.first, skip);
        own_read<V>(sh.dbias + threadIdx.x * V, dbias);
#pragma unroll
        for (int k = 0; k < PI; ++k) {
            const int r = p.row + k * P::ROWS, t = tb + r;
            if (r >= TT || t >= p.te) continue;
            const int at = r * CT + p.first;
            F2 x[Q], du[Q], f[Q], e[Q];
            whole(sh.g, r, du);
            own_read<V>(sh.x + at, x);
            own_read<V>(sh.slope + at, f);
            own_read<V>(sh.q + r * WHOLE + p.first, e);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                e[q] = mul2(fma2(e[q], f2(kLn2), mul2(du[q], x[q])), f[q]);
                dbias[q] = add2(dbias[q], e[q]);
            }
            put_dt(t, e);
#pragma unroll
            for (int q = 0; q < Q; ++q) {  // dt du + skip w
                float d[2] = {}, w[2] = {};
#pragma unroll
                for (int v = 0; v < (V > 1 ? 2 : 1); ++v) {
                    const int i = r * DW + P::entry(p.first + 2 * q + v);
                    d[v] = sh.du[i].x, w[v] = sh.w[i];
                }
                e[q] = fma2(f2(d[0], d[1]), du[q], mul2(skip[q], f2(w[0], w[1])));
            }
            put_x(A.dx, t, e);
            if constexpr (GATE) {
                whole(sh.y, r, e);
                own_read<V>(sh.zf + at, f);
#pragma unroll
                for (int q = 0; q < Q; ++q) e[q] = mul2(fma2(skip[q], x[q], e[q]), f[q]);
                put_x(A.dz, t, e);
            }
        }
        own_write<V>(sh.dbias + threadIdx.x * V, dbias);
        float* out = A.parts_bc + (((long long)p.ct * A.B + p.b) * A.T + tb) * 2 * A.N;
        for (int i = threadIdx.x; i < 2 * TT * NP; i += NT) {
            const int kind = i / (TT * NP), j = i - kind * TT * NP, t = j / NP, n = j % NP;
            if (n >= A.N || tb + t >= p.te) continue;
            float v = sh.sums[kind][0][j];
#pragma unroll
            for (int q = 1; q < W; ++q) v += sh.sums[kind][q][j];
            out[(long long)t * 2 * A.N + kind * A.N + n] = v;
        }
    };
    const int tiles = (p.te - p.t0 + TT - 1) / TT;
    for (int i = tiles - 1; i >= 0; --i) {
        const int tb = p.t0 + i * TT;
        __syncthreads();
        fetch(tb);  // on its way while the tile behind is finished
        if (i > 0) ahead(tb - TT);
        if (i + 1 < tiles) finish(tb + TT);
        prepare(tb);
        __syncthreads();
        F2 sA[2] = {f2(0.f), f2(0.f)};
        StateSums<L> sy, sg, sq;
        ChannelSums<L> sc;
        const float *vb = sh.b + order * VS + n0, *vc = sh.c + order * VS + n0;
        const float2* dtu = sh.du + entry;
        const float* ws = sh.w + entry;
        float *ys = sh.y + p.gl * CTP + p.c, *gs = sh.g + p.gl * CTP + p.c;  // the lane's parts
#pragma unroll 1
        for (int q = TT - SB; q >= 0; q -= SB) {
            F2 a[SB][2], hp[SB][2], h[2];
            mark(tb + q, h);
#pragma unroll
            for (int j4 = 0; j4 < SB; j4 += 4) {
                F2 u[4][2];
                decays<4, 4>(dtu + (q + j4) * DW, DW, vb + (q + j4) * NP, NP, A2, a + j4, u);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        hp[j4 + j][k] = h[k];
                        h[k] = fma2(a[j4 + j][k], h[k], u[j][k]);
                    }
            }
#pragma unroll
            for (int j = SB - 1; j >= 0; --j) {
                const int t = q + j;
                const float2 d = dtu[t * DW];
                const F2 dt = f2(d.x), u = f2(d.y), w = f2(ws[t * DW]);
                F2 bv[2], cv[2], dc[2], db[2], yy, dd, qq;
                read_vec<4>(vb + t * NP, bv);
                read_vec<4>(vc + t * NP, cv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    dc[k] = mul2(w, h[k]);
                    if constexpr (GATE) yy = k ? fma2(h[k], cv[k], yy) : mul2(h[k], cv[k]);
                    g[k] = fma2(w, cv[k], g[k]);
                    db[k] = mul2(u, g[k]);
                    dd = k ? fma2(g[k], bv[k], dd) : mul2(g[k], bv[k]);
                    g[k] = mul2(a[j][k], g[k]);
                    const F2 ah = mul2(g[k], hp[j][k]);
                    qq = k ? fma2(ah, A2[k], qq) : mul2(ah, A2[k]);
                    sA[k] = fma2(ah, dt, sA[k]);
                    h[k] = hp[j][k];
                }
                // j stands for t in the choice of what is handed on: q is a multiple of 4
                if constexpr (Sh::PARTS) {
                    if constexpr (GATE) ys[t * ROW] = total(yy);
                    gs[t * ROW] = total(dd);
                } else {
                    if constexpr (GATE) sy.add(sh.y + q * ROW, ROW, j, total(yy), p.lane, p.gl, p.c);
                    sg.add(sh.g + q * ROW, ROW, j, total(dd), p.lane, p.gl, p.c);
                }
                sq.add(sh.q + q * WHOLE, WHOLE, j, total(qq), p.lane, p.gl, p.c);
                sc.add(sh.sums[0][warp] + q * NP, sh.sums[1][warp] + q * NP, j, dc, db, p.lane, p.gl, p.cl);
            }
        }
        dA[0] = add2(dA[0], sA[0]), dA[1] = add2(dA[1], sA[1]);  // tile by tile: short sums lose less
    }
    __syncthreads();
    if (tiles > 0) finish(p.t0);
    const F2 zero[Q] = {};
    for (int t = p.te + p.row; t < p.t1; t += P::ROWS) {  // behind the sequence's end
        put_x(A.dx, t, zero);
        put_dt(t, zero);
        if constexpr (GATE) put_x(A.dz, t, zero);
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
    __syncthreads();
    if (p.row == 0) {  // the sums over tokens per channel: row by row, in order
        F2 dskip[Q], dbias[Q], o[Q];
        own_read<V>(sh.dskip + threadIdx.x * V, dskip);
        own_read<V>(sh.dbias + threadIdx.x * V, dbias);
        for (int r = 1; r < P::ROWS; ++r) {
            own_read<V>(sh.dskip + (r * P::QUADS + threadIdx.x) * V, o);
#pragma unroll
            for (int q = 0; q < Q; ++q) dskip[q] = add2(dskip[q], o[q]);
            own_read<V>(sh.dbias + (r * P::QUADS + threadIdx.x) * V, o);
#pragma unroll
            for (int q = 0; q < Q; ++q) dbias[q] = add2(dbias[q], o[q]);
        }
        store<false, float, V>(A.parts_ch + seg * 2 * A.E + p.column(), dskip, pw);
        store<false, float, V>(A.parts_ch + seg * 2 * A.E + A.E + p.column(), dbias, pw);
    }
}

// What the CTAs have left in the workspace, in one launch. The first `most` CTAs: db and dc from the channel tiles' sums, in their order. Such a
// CTA has `tokens` of a sequence; its threads stand for the 2 N values of a token's group, padded to a power of two (width), and as many
// groups at once as are left. The others: dA, dskip and ddt_bias from the sequences' and segments' sums, 32 columns and 8 slices of these
// per CTA, slices added up in order.
template <class XT>
__global__ void __launch_bounds__(256) sums_kernel(const SelArgs A, int width, int tokens, int most) {
    if ((int)blockIdx.x >= most) {
        __shared__ float sum[8][33];
        const long long EN = (long long)A.E * A.N, i = (long long)((int)blockIdx.x - most) * 32 + (threadIdx.x & 31);
        const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
        const bool in = i < sel_columns(A.E, A.N), ch = i >= EN;
        const float* from = ch ? A.parts_ch + (i - EN) : A.parts_A + i;
        const long long step = ch ? 2LL * A.E : EN;
        float v = 0.f;
        if (in)
#pragma unroll 4
            for (int k = slice; k < A.B * A.nseg; k += 8) v += from[k * step];
        sum[slice][lane] = v;
        __syncthreads();
        if (slice || !in) return;
        for (int k = 1; k < 8; ++k) v += sum[k][lane];
        if (!ch) A.dA[i] = v;
        else if (i - EN < A.E) {
            if (A.dskip) A.dskip[i - EN] = v;
        } else if (A.ddt_bias) {
            A.ddt_bias[i - EN - A.E] = v;
        }
        return;
    }
    const int n2 = 2 * A.N, per = (A.T + tokens - 1) / tokens, b = blockIdx.x / per, t0 = (blockIdx.x - b * per) * tokens;
    const int m = threadIdx.x & (width - 1), kind = m >= A.N, n = m - kind * A.N, step = 256 / width;
    if (m >= n2) return;
    const int len = A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T, rows = min(tokens, A.T - t0) * A.G;
    const long long all = (long long)A.B * A.T * n2, bt0 = (long long)b * A.T + t0;
    XT* to = static_cast<XT*>(kind ? A.db : A.dc) + bt0 * A.G * A.N + n;
    for (int r = threadIdx.x / width; r < rows; r += step) {
        const int t = A.G == 1 ? r : r / A.G, g = r - t * A.G;
        float v = 0.f;
        if (t0 + t < len) {
            const float* from = A.parts_bc + (long long)g * A.tiles * all + (bt0 + t) * n2 + m;
#pragma unroll 8
            for (int k = 0; k < A.tiles; ++k) v += from[k * all];
        }
        put(to + (long long)r * A.N, v);
    }
}

}  // namespace selective
}  // namespace lattice

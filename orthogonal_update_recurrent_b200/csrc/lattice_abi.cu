// lattice_abi.cu -- extern "C" entry points of liblattice (declared in
// include/lattice.h): argument checks and kernel choice. The launches live in one
// translation unit per kernel family (tu_*.cu, through launch.h).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "launch.h"
#include "waits.cuh"

using namespace lattice;

namespace {

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

Span span(const void* p, size_t bytes) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + bytes};
}
bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool dtype_ok(lattice_dtype t) { return t == LATTICE_F32 || t == LATTICE_BF16; }
size_t dsize(lattice_dtype t) { return t == LATTICE_BF16 ? 2 : 4; }
bool d_supported(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

thread_local char g_last_error[256] = "";

}  // namespace

namespace lattice {

// SMs of the current device (148 on B200; also the answer without a device).
int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
        return n;
    cudaGetLastError();  // clear the error of a host without a device
    return 148;
}

lattice_status cuda_fail(cudaError_t e) {
    cudaGetLastError();  // reported here, and not again by the next call's launch_status
    snprintf(g_last_error, sizeof(g_last_error), "%s: %s", cudaGetErrorName(e), cudaGetErrorString(e));
    return LATTICE_ERR_CUDA;
}

lattice_status launch_status() {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? LATTICE_OK : cuda_fail(e);
}

// CTAs per sequence for the CUDA-core scans: when the batch has fewer sequences than
// SMs, a cluster of G CTAs per sequence covers more of the device (G at most 4, at
// least 4 and at most 32 slots per CTA); otherwise 1. Measured on B200: 8-CTA clusters
// (8 slots per CTA) ran the long-context backward at half the speed of 4-CTA ones.
int cluster_split(int B, int H, int m) {
    const long long seqs = (long long)B * H;
    long long G = sm_count() / seqs;
    if (G > 4) G = 4;
    if (G > (m + 3) / 4) G = (m + 3) / 4;
    if (G < 2 || (m + G - 1) / G > 32) return 1;
    return (int)G;
}

}  // namespace lattice

namespace {

// ---- backward
constexpr int kBwdMaxM = 128;  // slots per head of the backward kernels

int bwd_seg(int chunk, int seg) {
    if (seg == 0) return chunk >= 64 ? chunk : chunk * ((64 + chunk - 1) / chunk);
    return (seg > 0 && seg % chunk == 0) ? seg : -1;
}

// CTAs per sequence of the backward kernel (see cluster_split).
int bwd_split(int B, int H, int m) { return cluster_split(B, H, m); }

// One warp waits, with the library's bounded wait, on an mbarrier that nothing ever
// arrives on: after limit_ns the wait gives up, sets the device status word and the
// kernel returns. Used to check, on a live GPU, that a wait that runs out is reported
// on the host and leaves the context usable.
__global__ void bounded_wait_selftest_kernel(unsigned long long limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    const uint32_t b = ptx::smem_u32(&bar);
    if (threadIdx.x == 0) {
        ptx::mbar_init(b, 1);
        abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    tc_wait(b, 0, &abort_flag, limit_ns);
}

lattice_status check_dims(int B, int H, int m, int d) {
    if (B < 1 || H < 1 || m < 1 || d < 1) return LATTICE_ERR_INVALID_ARG;
    if ((long long)B * H > 0x7fffffffLL) return LATTICE_ERR_UNSUPPORTED;
    if (!d_supported(d) || m > kMaxM) return LATTICE_ERR_UNSUPPORTED;
    return LATTICE_OK;
}

// ---- gated recurrence and block norms: fp16 is a type too, and rows may be strided
size_t type_size(lattice_dtype t) { return t == LATTICE_F32 ? 4 : 2; }
bool type_ok(lattice_dtype t) { return t == LATTICE_F32 || t == LATTICE_BF16 || t == LATTICE_F16; }

// Bytes from the first to the last element of [B][T] rows of C elements with these strides;
// false for a negative stride or an extent beyond 2^62 bytes.
bool strided_span(const void* p, size_t size, long long B, long long T, long long C, long long bs, long long ts,
                  Span* s) {
    if (bs < 0 || ts < 0) return false;
    const __int128 bytes = T < 1 ? 0 : ((__int128)(B - 1) * bs + (__int128)(T - 1) * ts + C) * size;
    if (bytes > ((__int128)1 << 62)) return false;
    *s = span(p, (size_t)bytes);
    return true;
}

// Whether an output overlaps an input or another output. in_same == out_same: the one pair
// that may be the same buffer.
bool clash(const Span* ins, int ni, const Span* outs, int no, const void* in_same, const void* out_same) {
    const uintptr_t same = in_same && in_same == out_same ? reinterpret_cast<uintptr_t>(in_same) : 0;
    for (int i = 0; i < no; ++i) {
        for (int k = 0; k < ni; ++k)
            if (overlap(outs[i], ins[k]) &&
                !(same && outs[i].lo == same && ins[k].lo == same && outs[i].hi == ins[k].hi))
                return true;
        for (int k = i + 1; k < no; ++k)
            if (overlap(outs[i], outs[k])) return true;
    }
    return false;
}

lattice_status check_gated(lattice_dtype x_dtype, lattice_dtype z_dtype, int z_per_head, int B, int T, int H, int d,
                           lattice_gate gate, lattice_write write, float tau) {
    if (B < 1 || T < 0 || H < 1 || d < 1 || !type_ok(x_dtype) || !type_ok(z_dtype)) return LATTICE_ERR_INVALID_ARG;
    if (gate != LATTICE_GATE_VALUE && gate != LATTICE_GATE_LOGIT) return LATTICE_ERR_INVALID_ARG;
    if (write != LATTICE_WRITE_PLAIN && write != LATTICE_WRITE_LEAKY && write != LATTICE_WRITE_UNIT)
        return LATTICE_ERR_INVALID_ARG;
    if (gate == LATTICE_GATE_LOGIT && !(tau > 0.f && tau < 3.4e38f)) return LATTICE_ERR_INVALID_ARG;
    if (z_dtype != LATTICE_F32 && z_dtype != x_dtype) return LATTICE_ERR_UNSUPPORTED;
    if ((long long)H * d > kGatedMaxSize || T > kGatedMaxSize) return LATTICE_ERR_UNSUPPORTED;
    if (z_per_head && !d_supported(d)) return LATTICE_ERR_UNSUPPORTED;
    return LATTICE_OK;
}

// The polynomial in t that meets (1 - (1 + t)^-tau)/t at the Chebyshev nodes of [0, 1], for
// tau <= 1; larger tau are halved first. It is off by at most 5e-8 of its value (tau = 1). With
// its coefficients rounded to fp32, of which they are up to 14 times the value together, and summed
// in fp32, 1 - a is off by up to 4e-7 of itself (1.2e-7 to 4e-7 over tau from 0.001 to 1).
void gated_poly(GatedArgs& a) {
    constexpr int n = kGatedPoly;
    double tau = a.tau;
    for (a.squares = 0; tau > 1; ++a.squares) tau /= 2;
    const double pi = 3.14159265358979323846;
    double f[n], cheb[n], c[n] = {}, prev[n] = {}, cur[n] = {};
    for (int k = 0; k < n; ++k) {
        const double t = 0.5 + 0.5 * cos(pi * (k + 0.5) / n);
        f[k] = -expm1(-tau * log1p(t)) / t;
    }
    for (int j = 0; j < n; ++j) {
        double s = 0;
        for (int k = 0; k < n; ++k) s += f[k] * cos(pi * j * (k + 0.5) / n);
        cheb[j] = s * (j ? 2.0 : 1.0) / n;
    }
    // T_0 = 1, T_1 = x, T_{j+1} = 2 x T_j - T_{j-1} with x = 2 t - 1, in powers of t
    prev[0] = 1, cur[0] = -1, cur[1] = 2;
    for (int j = 0; j < n; ++j) {
        for (int k = 0; k < n; ++k) c[k] += cheb[j] * (j ? cur[k] : prev[k]);
        if (j == 0) continue;
        double next[n];
        for (int k = 0; k < n; ++k) next[k] = (k ? 4 * cur[k - 1] : 0) - 2 * cur[k] - prev[k];
        for (int k = 0; k < n; ++k) prev[k] = cur[k], cur[k] = next[k];
    }
    for (int k = 0; k < n; ++k) {
        const float v = (float)c[k];
        uint32_t bits;
        memcpy(&bits, &v, 4);
        a.poly[k] = (unsigned long long)bits << 32 | bits;
    }
}

int gated_form(lattice_gate gate, lattice_write write, float tau) {
    return 3 * (gate == LATTICE_GATE_VALUE ? 0 : tau == 1.f ? 1 : 2) + (int)write;
}

// Whether the contiguous arrays of a gated call, whichever it has, and the channels suit
// vectors of v elements of x's size, and of fp32.
bool gated_vec(const GatedArgs& a, size_t size, size_t v) {
    return a.C % v == 0 && aligned(a.y, v * size) && aligned(a.dx, v * size) && aligned(a.h0, 4 * v) &&
           aligned(a.h_out, 4 * v) && aligned(a.dh_T, 4 * v) && aligned(a.dh0, 4 * v);
}
// Whether the rows at p do.
bool rows_vec(const void* p, size_t size, int B, int T, long long bs, long long ts, size_t bytes) {
    return aligned(p, bytes) && (B == 1 || bs * size % bytes == 0) && (T <= 1 || ts * size % bytes == 0);
}
// Whether every token's 16-bit gates per head are whole 32-bit words.
bool gate_words(const void* z, int H, long long bs, long long ts) {
    return aligned(z, 4) && H % 2 == 0 && bs % 2 == 0 && ts % 2 == 0;
}

// The layer operators' units, by type of x or of the call, that a call has launched or captured
// kernels of. Only these can have set their status word, and reading one takes 12 us.
enum LayerUnit { kGatedFwdUnit, kGatedBwdUnit, kNormUnit, kLayerNormUnit };
std::atomic<bool> g_unit_used[4][3];
void use_unit(LayerUnit u, lattice_dtype t) { g_unit_used[u][t].store(true, std::memory_order_relaxed); }
bool unit_used(LayerUnit u, lattice_dtype t) { return g_unit_used[u][t].load(std::memory_order_relaxed); }

template <class F>
lattice_status with_x(lattice_dtype t, F f) {
    return t == LATTICE_F32 ? f(0.f) : t == LATTICE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

// ---- block norms
// What both directions check, and the inputs they share, into a.
lattice_status check_norm(NormArgs& a, const void* y, lattice_dtype y_dtype, long long ys, const void* gate, long long gs,
                          const void* residual, lattice_dtype r_dtype, long long rs, const void* w_post, const void* w_pre,
                          lattice_dtype w_dtype, lattice_dtype dtype, long long N, int G, int D, lattice_act act, int post,
                          float scale, float eps) {
    if (!type_ok(dtype) || !type_ok(y_dtype) || !type_ok(r_dtype) || !type_ok(w_dtype)) return LATTICE_ERR_INVALID_ARG;
    if (N < 0 || G < 1 || D < 1 || N % G || ys < 0 || gs < 0 || rs < 0) return LATTICE_ERR_INVALID_ARG;
    if ((int)act < 0 || (int)act > 3 || (gate && act == LATTICE_ACT_NONE)) return LATTICE_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !(eps < 3.4e38f) || scale != scale) return LATTICE_ERR_INVALID_ARG;
    if (D > kNormMaxD || N > 0x7fffffffLL || ys > kNormMaxStride || gs > kNormMaxStride || rs > kNormMaxStride)
        return LATTICE_ERR_UNSUPPORTED;
    if ((y_dtype != LATTICE_F32 && y_dtype != dtype) || (residual && r_dtype != LATTICE_F32 && r_dtype != dtype) ||
        ((w_post || w_pre) && w_dtype != LATTICE_F32 && w_dtype != dtype))
        return LATTICE_ERR_UNSUPPORTED;
    if (N > 0 && !y) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(y, type_size(y_dtype)) || !aligned(gate, type_size(dtype)) || !aligned(residual, type_size(r_dtype)) ||
        !aligned(w_post, type_size(w_dtype)) || !aligned(w_pre, type_size(w_dtype)))
        return LATTICE_ERR_INVALID_ARG;
    a = NormArgs{};
    a.y = y; a.gate = gate; a.residual = residual; a.w_post = w_post; a.w_pre = w_pre;
    a.ys = (unsigned)ys; a.gs = (unsigned)gs; a.rs = (unsigned)rs;
    a.N = N; a.G = G; a.D = D; a.act = (int)act;
    a.scale = scale; a.eps = eps; a.inv_d = 1.f / (float)D; a.inv_d_rest = (float)(1. / D - (double)a.inv_d);
    a.post = post != 0;
    a.y32 = y_dtype == LATTICE_F32; a.r32 = r_dtype == LATTICE_F32; a.w32 = w_dtype == LATTICE_F32;
    return LATTICE_OK;
}
// Whether vectors of 8 elements read these rows: 16-byte pieces of a 16-bit type.
bool norm_rows_vec(const void* p, lattice_dtype t, long long N, int G, long long stride) {
    return aligned(p, 16) && (N <= G || stride * (long long)type_size(t) % 16 == 0);
}
// Whether row i starts i D mod 8 elements past a 16-byte boundary, with every row behind the one
// before it: then vectors may start before their row does (null: no such rows).
bool norm_rows_shift(const void* p, lattice_dtype t, long long N, int G, int D, long long stride) {
    const long long more = stride - (long long)G * D;
    return !p || (aligned(p, 16) && (N <= G || (more >= 0 && more * (long long)type_size(t) % 16 == 0)));
}
bool group_span(const void* p, lattice_dtype t, long long N, int G, int D, long long stride, Span* s) {
    return strided_span(p, type_size(t), N / G, 1, (long long)G * D, stride, 0, s) || !p;
}

// ---- short convolution
lattice_status check_conv(lattice_dtype x_dtype, lattice_dtype w_dtype, int B, int T, int C, int K, lattice_act act) {
    if (B < 1 || T < 0 || C < 1 || K < 1 || !type_ok(x_dtype) || !type_ok(w_dtype)) return LATTICE_ERR_INVALID_ARG;
    if ((int)act < 0 || (int)act > 3) return LATTICE_ERR_INVALID_ARG;
    if (act != LATTICE_ACT_NONE && act != LATTICE_ACT_SILU) return LATTICE_ERR_UNSUPPORTED;
    if (w_dtype != LATTICE_F32 && w_dtype != x_dtype) return LATTICE_ERR_UNSUPPORTED;
    if (K > kConvMaxK || C > kConvMaxSize || T > kConvMaxSize) return LATTICE_ERR_UNSUPPORTED;
    return LATTICE_OK;
}
// Channels per thread: as many as every row, output and weight can be read and written in vectors of
int conv_width(const ConvArgs& a, size_t sx, size_t sw) {
    for (int V = 4; V > 1; V /= 2) {
        const size_t v = V * sx;
        if (a.C % V == 0 && rows_vec(a.x, sx, a.B, a.T, a.xbs, a.xts, v) && (!a.dy || rows_vec(a.dy, sx, a.B, a.T, a.ybs, a.yts, v)) &&
            aligned(a.y, v) && aligned(a.state, v) && aligned(a.state_out, v) && aligned(a.dx, v) && aligned(a.dstate, v) &&
            aligned(a.dstate_out, v) && aligned(a.w, V * sw) && aligned(a.bias, V * sw))
            return V;
    }
    return 1;
}
// Tokens of a thread's run: those with which the waves of CTAs that the device holds at once take the fewest tokens one after
// the other, the inputs that a run reads beside its own and its start (as long as some 8 tokens) among them. (8 x 4096 tokens of 2048 bf16
// channels, 4 taps, forward: 1024 CTAs of 64 tokens, in 2.3 waves, 66 us.)
int conv_run(long long B, int T, int C, int K, bool bwd, int V) {
    const long long lanes = B * (C / V), held = (long long)sm_count() * conv_resident(bwd, K);
    const int beside = (bwd ? 3 : 1) * (K - 1) + 8;
    int best = 8;
    long long least = -1;
    for (int run = 8; run <= kConvMostRun; run += 8) {
        const long long ctas = (lanes * ((T + (long long)run - 1) / run) + 255) / 256, cost = (ctas + held - 1) / held * (run + beside);
        if (least < 0 || cost <= least) least = cost, best = run;
    }
    return best;
}
size_t conv_workspace(int B, int T, int C, int K) {  // for any width of a thread's channels
    int run = kConvMostRun;
    for (int V = 1; V <= 4; V *= 2) {
        const int r = C % V ? run : conv_run(B, T, C, K, true, V);
        run = r < run ? r : run;
    }
    return (size_t)B * (((size_t)T + run - 1) / run) * (K + 1) * C * 4;
}
void conv_args(ConvArgs& a, const void* x, lattice_dtype x_dtype, long long xbs, long long xts, const void* w, const void* bias,
               lattice_dtype w_dtype, const void* state, const int* lengths, int B, int T, int C, int K, lattice_act act) {
    a = ConvArgs{};
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.lengths = lengths;
    a.xbs = xbs; a.xts = xts;
    a.B = B; a.T = T; a.C = C; a.K = K; a.w32 = w_dtype == LATTICE_F32; a.silu = act == LATTICE_ACT_SILU;
}

// ---- selective scan
struct SelPlan {
    int S, W, tiles, nseg, seg;
};
// Channel tiles of a group
long long sel_tiles(int Eg, int lanes, int W) {
    const int per = W * (32 / lanes);
    return ((long long)Eg + per - 1) / per;
}
// Warps of a CTA: 8, or 2 where 8 would leave so many more of them without channels that it pays: a warp of two takes 1.1 times the time,
// backward, with its share of the sums over channels, 1.5 times (mid-size layer: 614 and 672 us, 1635 and 2446 us; 20 sequences of 49370
// tokens, 12 channels, 16 states: 916 us with 8 warps and 283 us with 2, backward 1822 and 742 us). Backward, two have to be ahead by 1.7:
// from 1.5 on (groups of 65 to 80 channels at 16 states, 33 to 40 at 32) neither is always. 72 channels, 32 sequences of 2048 tokens, 74 of
// 1024, 148 of 1024, 300 of 512: 522 / 276 / 429 / 520 us with 8 and 489 / 314 / 425 / 498 us with 2; 36 channels, 32 states: 563 and 635 us.
int sel_warps(int Eg, int lanes, bool bwd) {
    return (double)sel_tiles(Eg, lanes, 8) * 4 > (bwd ? 1.7 : 1.1) * (double)sel_tiles(Eg, lanes, 2) ? 2 : 8;
}
// How the work is spread. A CTA has 256/L channels (64/L for few channels) with N padded to L S states, and goes through its tokens alone.
// With few CTAs the device is filled by two states per lane instead of four (twice the CTAs), or by segments of the time axis, whose states
// take a pass of their own (its exponentials are the forward pass's again). The times below, in us per token of a CTA's and by CTAs per
// SM, are what was measured with CTAs of 8 warps (bf16, 16 states, gate); the cheapest is taken. Forward,
// 1024 / 2048 / 4096 / 8192 / 16384 channels of 4096, 4096, 2048, 2048, 2048 tokens: four states 430 / 435 / 238 / 238 / 355 us, two states
// 297 / 297 / 167 / 240 / 427, segments 111 / 170 / 181 / 312; backward, whole 1155 / 1201 / 627 / 637 / 865, segments 188 / 303 / 329 / 589.
// They stand for the other forms too, whose CTAs have as many states, and are right there as long as an SM holds as many of them. Backward it
// does not always: of CTAs with 65 to 128 states per channel one instead of two (4 x 2048 tokens of 256 channels, 128 states: two segments
// are taken, 941 us, whole sequences 839 us), of CTAs of two warps 4 to 7 instead of 8 (16 x 2048 tokens, two groups of 6 channels: 32
// segments are taken, 87 us, 24 segments 78 us).
SelPlan sel_plan(int B, int T, int E, int N, int G, bool bwd) {
    const int np = sel_padded(N), Eg = E / G;
    const long long sm = sm_count(), tiles = ((long long)T + kSelTile - 1) / kSelTile;
    const double whole[2][3] = {{0.11, 0.165, 0.08}, {0.30, 0.39, 0.205}}, split[2][3] = {{0.168, 0.26, 0.13}, {0.37, 0.565, 0.29}},
                 two[3] = {0.072, 0.117, 0.052};  // one CTA per SM, two, and each of more
    SelPlan p = {};
    double best = -1;
    auto offer = [&](int S, bool segments, const double* us) {
        const int W = sel_warps(Eg, np / S, bwd), unit = 8 / W;  // CTAs that count as one of 8 warps' channels
        const long long ct = sel_tiles(Eg, np / S, W), base = (long long)B * G * ct;
        long long n = 1, tokens = T;
        if (segments) {
            n = 2 * sm * unit / base;
            if (n > tiles / 4) n = tiles / 4;
            if (n <= 1) return;
            tokens = (tiles + n - 1) / n * kSelTile;
            n = (T + tokens - 1) / tokens;
        }
        const long long per = (base * n + sm * unit - 1) / (sm * unit);
        const double time = (double)tokens * (per <= 2 ? us[per - 1] : us[2] * (double)per) + (segments ? 15 : 0);
        if (best < 0 || time < best) best = time, p = {S, W, (int)ct, (int)n, (int)(tokens > 0 ? tokens : 1)};
    };
    offer(4, false, whole[bwd]);
    offer(4, true, split[bwd]);
    if (!bwd && np <= 32) offer(2, false, two);
    return p;
}
// Floats of the workspace's parts, each a multiple of 4: the segments' states and sums, and backward the CTAs' sums
struct SelSpace {
    size_t state, sum, A, ch, bc;
    size_t bytes() const { return 4 * (state + sum + A + ch + bc); }
};
SelSpace sel_space(const SelPlan& p, int B, int T, int E, int N, int G, bool bwd) {
    auto four = [](size_t n) { return (n + 3) / 4 * 4; };
    const size_t rows = (size_t)B * p.nseg;
    SelSpace s = {};
    if (p.nseg > 1) s.state = four(rows * E * N), s.sum = four(rows * E);
    if (bwd) s.A = four(rows * E * N), s.ch = four(rows * 2 * E), s.bc = four((size_t)G * p.tiles * B * T * 2 * N);
    return s;
}
lattice_status check_selective(lattice_dtype x_dtype, lattice_dtype dt_dtype, int B, int T, int E, int N, int G) {
    if (B < 1 || T < 0 || E < 1 || N < 1 || G < 1 || E % G || !type_ok(x_dtype) || !type_ok(dt_dtype)) return LATTICE_ERR_INVALID_ARG;
    if (dt_dtype != LATTICE_F32 && dt_dtype != x_dtype) return LATTICE_ERR_UNSUPPORTED;
    if (N > kSelMaxN || E > kSelMaxSize || T > kSelMaxSize) return LATTICE_ERR_UNSUPPORTED;
    return LATTICE_OK;
}
// What the calls share: their inputs, checked, into a, and their spans.
struct SelInputs {
    Span s[10];
    int n;
};
lattice_status sel_inputs(SelArgs& a, SelInputs& in, const void* x, lattice_dtype x_dtype, long long xbs, long long xts, const void* dt,
                          lattice_dtype dt_dtype, long long dbs, long long dts, const float* A, const void* b, long long bbs,
                          long long bts, const void* c, long long cbs, long long cts, const float* skip, const void* z,
                          long long zbs, long long zts, const float* dt_bias, int softplus, const int* lengths, int B, int T, int E,
                          int N, int G) {
    const size_t sx = type_size(x_dtype), sd = type_size(dt_dtype);
    if (!A || (T > 0 && (!x || !dt || !b || !c))) return LATTICE_ERR_INVALID_ARG;
    Span s[5] = {};
    if (!strided_span(x, sx, B, T, E, xbs, xts, s) || !strided_span(dt, sd, B, T, E, dbs, dts, s + 1) ||
        !strided_span(b, sx, B, T, (long long)G * N, bbs, bts, s + 2) || !strided_span(c, sx, B, T, (long long)G * N, cbs, cts, s + 3) ||
        (z && !strided_span(z, sx, B, T, E, zbs, zts, s + 4)))
        return LATTICE_ERR_INVALID_ARG;
    for (const void* p : {x, b, c, z})
        if (!aligned(p, sx)) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(dt, sd) || !aligned(A, 4) || !aligned(skip, 4) || !aligned(dt_bias, 4) || !aligned(lengths, 4)) return LATTICE_ERR_INVALID_ARG;
    in.n = 0;
    for (const Span& v : s) in.s[in.n++] = v;
    in.s[in.n++] = span(A, (size_t)E * N * 4);
    in.s[in.n++] = span(skip, skip ? (size_t)E * 4 : 0);
    in.s[in.n++] = span(dt_bias, dt_bias ? (size_t)E * 4 : 0);
    in.s[in.n++] = span(lengths, lengths ? (size_t)B * 4 : 0);
    a = SelArgs{};
    a.x = x; a.dt = dt; a.z = z; a.b = b; a.c = c; a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.lengths = lengths;
    a.xbs = xbs; a.xts = xts; a.dbs = dbs; a.dts = dts; a.zbs = zbs; a.zts = zts; a.bbs = bbs; a.bts = bts; a.cbs = cbs; a.cts = cts;
    a.B = B; a.T = T; a.E = E; a.N = N; a.G = G; a.Eg = E / G;
    a.nmarks = (int)((T + (long long)kSelMark - 1) / kSelMark);
    a.dt32 = dt_dtype == LATTICE_F32; a.softplus = softplus != 0;
    a.vec_n = N % 4 == 0 && aligned(A, 16);
    return LATTICE_OK;
}
// Whether rows of channels and their outputs can be read and written in vectors of V, a sequence of each within 2^31 bytes
bool sel_vec(const SelArgs& a, size_t sx, int V) {
    const size_t sd = a.dt32 ? 4 : sx, bx = V * sx, bd = V * sd;
    for (long long ts : {a.xts, a.dts, a.zts, a.bts, a.cts, a.yts, (long long)a.E})
        if (((__int128)a.T * ts + a.E + (long long)a.G * a.N) * 4 > 0x7fffffffLL) return false;
    return a.Eg % V == 0 && rows_vec(a.x, sx, a.B, a.T, a.xbs, a.xts, bx) && rows_vec(a.dt, sd, a.B, a.T, a.dbs, a.dts, bd) &&
           (!a.z || rows_vec(a.z, sx, a.B, a.T, a.zbs, a.zts, bx)) && (!a.dy || rows_vec(a.dy, sx, a.B, a.T, a.ybs, a.yts, bx)) &&
           aligned(a.y, bx) && aligned(a.dx, bx) && aligned(a.dz, bx) && aligned(a.ddt, bd);
}
void sel_place(SelArgs& a, const SelPlan& p, const SelSpace& s, void* workspace) {
    a.tiles = p.tiles; a.nseg = p.nseg; a.seg = p.seg;
    a.joined = p.nseg > kSelFold || (p.nseg > 1 && a.h0 && a.h0 == a.h_out);  // in place: h0 is read before any CTA writes
    float* w = static_cast<float*>(workspace);
    if (p.nseg > 1) a.seg_state = w, a.seg_sum = w + s.state;
    if (s.A) a.parts_A = w + s.state + s.sum, a.parts_ch = a.parts_A + s.A, a.parts_bc = a.parts_ch + s.ch;
}

}  // namespace

extern "C" {

int lattice_version(void) { return 100; }

const char* lattice_status_string(lattice_status s) {
    switch (s) {
        case LATTICE_OK: return "ok";
        case LATTICE_ERR_INVALID_ARG: return "invalid argument";
        case LATTICE_ERR_UNSUPPORTED: return "unsupported size or dtype";
        case LATTICE_ERR_CUDA: return "CUDA error";
        case LATTICE_ERR_TIMEOUT: return "device-side wait timed out";
    }
    return "unknown status";
}

lattice_impl lattice_chunk_impl(int B, int H, int m, int d, int chunk_size, lattice_dtype x_dtype,
                                lattice_dtype q_dtype) {
    if (chunk_size <= 1) return LATTICE_IMPL_SIMT;
    const bool xb = x_dtype == LATTICE_BF16, qb = q_dtype == LATTICE_BF16;
    if (tc_supported(LATTICE_IMPL_SPLIT_REG, m, d, chunk_size, xb, qb) && B >= 1 && H >= 1 &&
        (long long)B * H <= reg_cluster_capacity(d))
        return LATTICE_IMPL_SPLIT_REG;
    if (tc_supported(LATTICE_IMPL_TCGEN05, m, d, chunk_size, xb, qb)) return LATTICE_IMPL_TCGEN05;
    return LATTICE_IMPL_SIMT;
}

lattice_status lattice_scan_fwd_ex(const void* x, lattice_dtype x_dtype, const float* c,
                                   const void* q, lattice_dtype q_dtype, const float* mu,
                                   const float* eta, const float* S0, float* S_out, float* y,
                                   int B, int T, int H, int m, int d, int chunk_size,
                                   lattice_mode mode, lattice_chunk_form form, lattice_impl impl,
                                   void* stream) {
    if ((int)form < 0 || (int)form > 3) return LATTICE_ERR_INVALID_ARG;
    const bool lin1 = ((int)form & LATTICE_CHUNK_LIN1) != 0;
    const bool cnorm = ((int)form & LATTICE_CHUNK_NORM_AT_BOUNDARY) != 0;
    if (B < 1 || H < 1 || m < 1 || d < 1 || T < 0 || chunk_size < 1) return LATTICE_ERR_INVALID_ARG;
    if (!dtype_ok(x_dtype) || !dtype_ok(q_dtype)) return LATTICE_ERR_INVALID_ARG;
    if (impl != LATTICE_IMPL_AUTO && impl != LATTICE_IMPL_SIMT && impl != LATTICE_IMPL_TCGEN05 &&
        impl != LATTICE_IMPL_TCGEN05_SPLIT && impl != LATTICE_IMPL_SPLIT_REG &&
        impl != LATTICE_IMPL_SPLIT_REG8)
        return LATTICE_ERR_INVALID_ARG;
    if (mode != LATTICE_SIM && mode != LATTICE_DEC) return LATTICE_ERR_INVALID_ARG;
    const bool dec = mode == LATTICE_DEC;
    lattice_status ds = check_dims(B, H, m, d);
    if (ds != LATTICE_OK) return ds;
    if (!S0 || !S_out) return LATTICE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !c || !q || !mu || !y)) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(S0, 16) || !aligned(S_out, 16)) return LATTICE_ERR_INVALID_ARG;
    const size_t nS = (size_t)B * H * m * d * 4;
    const Span sS0 = span(S0, nS), sSo = span(S_out, nS);
    if (S0 != S_out && overlap(sS0, sSo)) return LATTICE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (S0 != S_out) {
            cudaError_t e = cudaMemcpyAsync(S_out, S0, nS, cudaMemcpyDeviceToDevice, st);
            if (e != cudaSuccess) return cuda_fail(e);
        }
        return LATTICE_OK;
    }
    const size_t ntok = (size_t)B * T * H;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(c, 4) || !aligned(mu, 4) ||
        !aligned(q, dsize(q_dtype)) || (eta && !aligned(eta, 4)))
        return LATTICE_ERR_INVALID_ARG;
    const Span sx = span(x, ntok * d * dsize(x_dtype)), sc = span(c, ntok * m * 4),
               sq = span(q, ntok * m * dsize(q_dtype)), smu = span(mu, ntok * 4),
               seta = span(eta, eta ? ntok * 4 : 0), sy = span(y, ntok * d * 4);
    const Span ins[] = {sx, sc, sq, smu, seta, sS0};
    for (const Span& s : ins)
        if (overlap(s, sy) || (s.lo != sS0.lo && overlap(s, sSo))) return LATTICE_ERR_INVALID_ARG;
    if (overlap(sy, sSo)) return LATTICE_ERR_INVALID_ARG;

    ScanArgs a{x, x_dtype == LATTICE_BF16, c, q, q_dtype == LATTICE_BF16, mu, eta, S0, S_out, y,
               B, T, H, m, chunk_size};
    const bool tc_choice = impl == LATTICE_IMPL_TCGEN05 || impl == LATTICE_IMPL_TCGEN05_SPLIT ||
                           impl == LATTICE_IMPL_SPLIT_REG || impl == LATTICE_IMPL_SPLIT_REG8;
    a.cnorm = cnorm && chunk_size > 1 ? 1 : 0;
    if (chunk_size == 1 && cnorm) {  // normalising after every token is the exact recurrence
        if (tc_choice) return LATTICE_ERR_UNSUPPORTED;
        return launch_scan_simt(a, d, false, dec, false, st);
    }
    if (chunk_size == 1 || dec || lin1 || cnorm) {  // the tensor-core kernels: Eq. 17, per-token normaliser, similarity objective
        if (tc_choice) return LATTICE_ERR_UNSUPPORTED;
        return launch_scan_simt(a, d, chunk_size > 1, dec, lin1, st);
    }
    if (impl == LATTICE_IMPL_AUTO) impl = lattice_chunk_impl(B, H, m, d, chunk_size, x_dtype, q_dtype);
    if (impl != LATTICE_IMPL_SIMT) {
        if (!tc_supported(impl, m, d, chunk_size, a.x_bf16, a.q_bf16)) return LATTICE_ERR_UNSUPPORTED;
        return launch_tc(impl, a, d, st);
    }
    return launch_scan_simt(a, d, true, false, false, st);
}

lattice_status lattice_scan_fwd_impl(const void* x, lattice_dtype x_dtype, const float* c,
                                     const void* q, lattice_dtype q_dtype, const float* mu,
                                     const float* eta, const float* S0, float* S_out, float* y,
                                     int B, int T, int H, int m, int d, int chunk_size,
                                     lattice_mode mode, lattice_impl impl, void* stream) {
    return lattice_scan_fwd_ex(x, x_dtype, c, q, q_dtype, mu, eta, S0, S_out, y, B, T, H, m, d,
                               chunk_size, mode, LATTICE_CHUNK_LIN2, impl, stream);
}

lattice_status lattice_scan_fwd(const void* x, lattice_dtype x_dtype, const float* c,
                                const void* q, lattice_dtype q_dtype, const float* mu,
                                const float* eta, const float* S0, float* S_out, float* y, int B,
                                int T, int H, int m, int d, int chunk_size, lattice_mode mode,
                                void* stream) {
    return lattice_scan_fwd_impl(x, x_dtype, c, q, q_dtype, mu, eta, S0, S_out, y, B, T, H, m, d,
                                 chunk_size, mode, LATTICE_IMPL_AUTO, stream);
}

lattice_status lattice_step(float* S, const void* x, lattice_dtype x_dtype, const float* c,
                            const void* q, lattice_dtype q_dtype, const float* mu,
                            const float* eta, float* y, int B, int H, int m, int d,
                            lattice_mode mode, void* stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(q_dtype)) return LATTICE_ERR_INVALID_ARG;
    if (mode != LATTICE_SIM && mode != LATTICE_DEC) return LATTICE_ERR_INVALID_ARG;
    const bool dec = mode == LATTICE_DEC;
    lattice_status ds = check_dims(B, H, m, d);
    if (ds != LATTICE_OK) return ds;
    if (!S || !x || !c || !q || !mu || !y) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(S, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(c, 4) ||
        !aligned(mu, 4) || !aligned(q, dsize(q_dtype)) || (eta && !aligned(eta, 4)))
        return LATTICE_ERR_INVALID_ARG;
    const size_t nbh = (size_t)B * H;
    const Span sS = span(S, nbh * m * d * 4), sy = span(y, nbh * d * 4);
    const Span ins[] = {span(x, nbh * d * dsize(x_dtype)), span(c, nbh * m * 4),
                        span(q, nbh * m * dsize(q_dtype)), span(mu, nbh * 4),
                        span(eta, eta ? nbh * 4 : 0)};
    for (const Span& s : ins)
        if (overlap(s, sS) || overlap(s, sy)) return LATTICE_ERR_INVALID_ARG;
    if (overlap(sS, sy)) return LATTICE_ERR_INVALID_ARG;
    StepArgs a{S, x, x_dtype == LATTICE_BF16, c, q, q_dtype == LATTICE_BF16, mu, eta, y, B, H, m};
    return launch_step(a, d, dec, static_cast<cudaStream_t>(stream));
}

lattice_status lattice_readout(const float* S, const void* q, lattice_dtype q_dtype, float* y,
                               int B, int H, int m, int d, void* stream) {
    if (!dtype_ok(q_dtype)) return LATTICE_ERR_INVALID_ARG;
    lattice_status ds = check_dims(B, H, m, d);
    if (ds != LATTICE_OK) return ds;
    if (!S || !q || !y) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(S, 16) || !aligned(y, 16) || !aligned(q, dsize(q_dtype))) return LATTICE_ERR_INVALID_ARG;
    const size_t nbh = (size_t)B * H;
    const Span sy = span(y, nbh * d * 4);
    if (overlap(sy, span(S, nbh * m * d * 4)) || overlap(sy, span(q, nbh * m * dsize(q_dtype))))
        return LATTICE_ERR_INVALID_ARG;
    ReadoutArgs a{S, q, q_dtype == LATTICE_BF16, y, B, H, m};
    return launch_readout(a, d, static_cast<cudaStream_t>(stream));
}

size_t lattice_scan_bwd_workspace_bytes(int B, int T, int H, int m, int d, int chunk_size,
                                        int seg_tokens) {
    if (B < 1 || H < 1 || m < 1 || d < 1 || T < 0 || chunk_size < 1) return 0;
    if (check_dims(B, H, m, d) != LATTICE_OK || m > kBwdMaxM) return 0;
    const int seg = bwd_seg(chunk_size, seg_tokens);
    if (seg < 1) return 0;
    const int G = bwd_split(B, H, m), spc = (m + G - 1) / G;
    const size_t tok = (size_t)B * H * G * bwd_ws_floats_per_seq(T, spc, d, seg) * sizeof(float);
    if (!chunk_bwd_supported(m, d, chunk_size)) return tok;
    // the chunk-parallel kernel serves the shape; the token kernel stays the fallback
    // for buffers it cannot read with vector loads, so the workspace covers both
    const size_t cb = chunk_bwd_ws_floats(B, T, H, m, d, chunk_size) * sizeof(float);
    return cb > tok ? cb : tok;
}

lattice_status lattice_scan_bwd(const void* x, lattice_dtype x_dtype, const float* c,
                                const void* q, lattice_dtype q_dtype, const float* mu,
                                const float* eta, const float* S0, const float* dy,
                                const float* dS_T, float* dx, float* dc, float* dq, float* dmu,
                                float* deta, float* dS0, void* workspace, size_t workspace_bytes,
                                int B, int T, int H, int m, int d, int chunk_size, int seg_tokens,
                                void* stream) {
    if (B < 1 || H < 1 || m < 1 || d < 1 || T < 0 || chunk_size < 1) return LATTICE_ERR_INVALID_ARG;
    if (!dtype_ok(x_dtype) || !dtype_ok(q_dtype)) return LATTICE_ERR_INVALID_ARG;
    lattice_status ds = check_dims(B, H, m, d);
    if (ds != LATTICE_OK) return ds;
    if (m > kBwdMaxM) return LATTICE_ERR_UNSUPPORTED;
    const int seg = bwd_seg(chunk_size, seg_tokens);
    if (seg < 1) return LATTICE_ERR_INVALID_ARG;
    const size_t need = lattice_scan_bwd_workspace_bytes(B, T, H, m, d, chunk_size, seg_tokens);
    if (!S0 || !dS0 || !workspace || workspace_bytes < need) return LATTICE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !c || !q || !mu || !dy || !dx || !dc || !dq || !dmu))
        return LATTICE_ERR_INVALID_ARG;
    if (!aligned(S0, 16) || !aligned(dS0, 16) || !aligned(workspace, 16) || (dS_T && !aligned(dS_T, 16)))
        return LATTICE_ERR_INVALID_ARG;
    const size_t ntok = (size_t)B * T * H, nS = (size_t)B * H * m * d * 4;
    if (T > 0 && (!aligned(x, dsize(x_dtype)) || !aligned(c, 4) || !aligned(mu, 4) || !aligned(q, dsize(q_dtype)) ||
                  !aligned(dy, 4) || !aligned(dx, 4) || !aligned(dc, 4) || !aligned(dq, 4) ||
                  !aligned(dmu, 4) || (eta && !aligned(eta, 4)) || (deta && !aligned(deta, 4))))
        return LATTICE_ERR_INVALID_ARG;
    float* deta_w = eta ? deta : nullptr;
    const size_t tb = T > 0 ? 1 : 0;  // token-indexed buffers are empty when T == 0
    const Span ins[] = {span(x, tb * ntok * d * dsize(x_dtype)), span(c, tb * ntok * m * 4),
                        span(q, tb * ntok * m * dsize(q_dtype)), span(mu, tb * ntok * 4),
                        span(eta, eta ? tb * ntok * 4 : 0), span(S0, nS),
                        span(dy, tb * ntok * d * 4), span(dS_T, dS_T ? nS : 0)};
    const Span outs[] = {span(dx, tb * ntok * d * 4), span(dc, tb * ntok * m * 4),
                         span(dq, tb * ntok * m * 4), span(dmu, tb * ntok * 4),
                         span(deta_w, deta_w ? tb * ntok * 4 : 0), span(dS0, nS),
                         span(workspace, need)};
    for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
        for (const Span& s : ins)
            if (overlap(outs[i], s)) return LATTICE_ERR_INVALID_ARG;
        for (size_t k = i + 1; k < sizeof(outs) / sizeof(outs[0]); ++k)
            if (overlap(outs[i], outs[k])) return LATTICE_ERR_INVALID_ARG;
    }
    // Chunks of 2..64 tokens: the chunk-parallel kernel, when x, dy and dx take 16-byte
    // vector accesses; otherwise (and for the exact recurrence) the token kernel.
    if (chunk_bwd_supported(m, d, chunk_size) &&
        (T == 0 || (aligned(x, 16) && aligned(dy, 16) && aligned(dx, 16)))) {
        const int G = chunk_bwd_ctas(m);
        BwdArgs a{x, x_dtype == LATTICE_BF16, c, q, q_dtype == LATTICE_BF16, mu, eta, S0, dy, dS_T,
                  dx, dc, dq, dmu, deta_w, dS0, static_cast<float*>(workspace), B, T, H, m, chunk_size,
                  seg, G, kCbSlots};
        return launch_chunk_bwd(a, d, static_cast<cudaStream_t>(stream));
    }
    const int G = bwd_split(B, H, m);
    BwdArgs a{x, x_dtype == LATTICE_BF16, c, q, q_dtype == LATTICE_BF16, mu, eta, S0, dy, dS_T,
              dx, dc, dq, dmu, deta_w, dS0, static_cast<float*>(workspace), B, T, H, m, chunk_size, seg,
              G, (m + G - 1) / G};
    return launch_bwd(a, d, static_cast<cudaStream_t>(stream));
}

lattice_status lattice_gated_scan_fwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride,
                                      long long x_token_stride, const void* z, lattice_dtype z_dtype,
                                      long long z_batch_stride, long long z_token_stride, int z_per_head,
                                      const float* h0, float* h_out, void* y, float* marks, const int* lengths,
                                      int B, int T, int H, int d, lattice_gate gate, lattice_write write,
                                      float tau, void* stream) {
    lattice_status s = check_gated(x_dtype, z_dtype, z_per_head, B, T, H, d, gate, write, tau);
    if (s != LATTICE_OK) return s;
    const long long C = (long long)H * d, Cz = z_per_head ? H : C, nm = (T + (long long)kGatedMark - 1) / kGatedMark;
    Span sx, sz;
    if (!strided_span(x, type_size(x_dtype), B, T, C, x_batch_stride, x_token_stride, &sx) ||
        !strided_span(z, type_size(z_dtype), B, T, Cz, z_batch_stride, z_token_stride, &sz))
        return LATTICE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !z || (!y && !marks))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(x, type_size(x_dtype)) || !aligned(z, type_size(z_dtype)) || !aligned(y, type_size(x_dtype)) ||
        !aligned(h0, 4) || !aligned(h_out, 4) || !aligned(marks, 16) || !aligned(lengths, 4))
        return LATTICE_ERR_INVALID_ARG;
    const size_t nh = (size_t)B * C * 4;
    const Span ins[] = {sx, sz, span(h0, h0 ? nh : 0), span(lengths, lengths ? (size_t)B * 4 : 0)};
    const Span outs[] = {span(h_out, h_out ? nh : 0), span(y, y ? (size_t)B * T * C * type_size(x_dtype) : 0),
                         span(marks, marks ? (size_t)B * nm * C * 4 : 0)};
    if (clash(ins, 4, outs, 3, h0, h_out)) return LATTICE_ERR_INVALID_ARG;
    GatedArgs a = {};
    a.x = x; a.z = z; a.h0 = h0; a.h_out = h_out; a.y = y; a.marks = marks; a.lengths = lengths;
    a.xbs = x_batch_stride; a.xts = x_token_stride; a.zbs = z_batch_stride; a.zts = z_token_stride;
    a.B = B; a.T = T; a.C = (int)C; a.d = d; a.nmarks = (int)nm; a.tau = tau;
    a.z32 = z_dtype == LATTICE_F32; a.zhead = z_per_head != 0;
    a.zwords = gate_words(z, H, a.zbs, a.zts);
    if (gate == LATTICE_GATE_LOGIT && tau != 1.f) gated_poly(a);
    const size_t sx_ = type_size(x_dtype), sz_ = type_size(z_dtype), v = kGatedFwdVec;
    const bool vec = gated_vec(a, sx_, v) && rows_vec(x, sx_, B, T, a.xbs, a.xts, v * sx_) &&
                     (a.zhead || rows_vec(z, sz_, B, T, a.zbs, a.zts, v * sz_));
    a.wide = vec && C % (16 / sx_) == 0 && rows_vec(x, sx_, B, T, a.xbs, a.xts, 16) &&
             (a.zhead || rows_vec(z, sz_, B, T, a.zbs, a.zts, 16));
    use_unit(kGatedFwdUnit, x_dtype);
    return with_x(x_dtype, [&](auto t) {
        return gated::launch_fwd<decltype(t)>(a, gated_form(gate, write, tau), vec, static_cast<cudaStream_t>(stream));
    });
}

size_t lattice_gated_scan_marks_bytes(int B, int T, int H, int d) {
    if (B < 1 || T < 0 || H < 1 || d < 1 || (long long)H * d > kGatedMaxSize || T > kGatedMaxSize) return 0;
    return (size_t)B * ((T + (size_t)kGatedMark - 1) / kGatedMark) * H * d * 4;
}

lattice_status lattice_gated_scan_bwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride,
                                      long long x_token_stride, const void* z, lattice_dtype z_dtype,
                                      long long z_batch_stride, long long z_token_stride, int z_per_head,
                                      const void* dy, long long dy_batch_stride, long long dy_token_stride,
                                      const float* marks, const float* dh_T, void* dx, void* dz, float* dh0,
                                      const int* lengths, int B, int T, int H, int d, lattice_gate gate,
                                      lattice_write write, float tau, void* stream) {
    lattice_status s = check_gated(x_dtype, z_dtype, z_per_head, B, T, H, d, gate, write, tau);
    if (s != LATTICE_OK) return s;
    const long long C = (long long)H * d, Cz = z_per_head ? H : C, nm = (T + (long long)kGatedMark - 1) / kGatedMark;
    const size_t sx_ = type_size(x_dtype), sz_ = type_size(z_dtype);
    Span sx, sz, sdy;
    if (!strided_span(x, sx_, B, T, C, x_batch_stride, x_token_stride, &sx) ||
        !strided_span(z, sz_, B, T, Cz, z_batch_stride, z_token_stride, &sz) ||
        !strided_span(dy, sx_, B, T, C, dy_batch_stride, dy_token_stride, &sdy))
        return LATTICE_ERR_INVALID_ARG;
    if (!dh0 || (T > 0 && (!x || !z || !dy || !marks || !dx || !dz))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(x, sx_) || !aligned(z, sz_) || !aligned(dy, sx_) || !aligned(dx, sx_) || !aligned(dz, sz_) ||
        !aligned(marks, 16) || !aligned(dh_T, 4) || !aligned(dh0, 4) || !aligned(lengths, 4))
        return LATTICE_ERR_INVALID_ARG;
    const size_t nh = (size_t)B * C * 4, nt = (size_t)B * T;
    const Span ins[] = {sx, sz, sdy, span(marks, T > 0 ? (size_t)B * nm * C * 4 : 0), span(dh_T, dh_T ? nh : 0),
                        span(lengths, lengths ? (size_t)B * 4 : 0)};
    const Span outs[] = {span(dx, nt * C * sx_), span(dz, nt * Cz * sz_), span(dh0, nh)};
    if (clash(ins, 6, outs, 3, nullptr, nullptr)) return LATTICE_ERR_INVALID_ARG;
    GatedArgs a = {};
    a.x = x; a.z = z; a.marks = const_cast<float*>(marks); a.lengths = lengths;
    a.dy = dy; a.dh_T = dh_T; a.dx = dx; a.dz = dz; a.dh0 = dh0;
    a.xbs = x_batch_stride; a.xts = x_token_stride; a.zbs = z_batch_stride; a.zts = z_token_stride;
    a.dybs = dy_batch_stride; a.dyts = dy_token_stride;
    a.B = B; a.T = T; a.C = (int)C; a.d = d; a.nmarks = (int)nm; a.tau = tau;
    a.z32 = z_dtype == LATTICE_F32; a.zhead = z_per_head != 0;
    a.zwords = gate_words(z, H, a.zbs, a.zts);
    if (gate == LATTICE_GATE_LOGIT && tau != 1.f) gated_poly(a);
    const size_t v = a.zhead ? kGatedHeadVec : kGatedBwdVec;
    const bool vec = gated_vec(a, sx_, v) && rows_vec(x, sx_, B, T, a.xbs, a.xts, v * sx_) &&
                     rows_vec(dy, sx_, B, T, a.dybs, a.dyts, v * sx_) &&
                     (a.zhead || (rows_vec(z, sz_, B, T, a.zbs, a.zts, v * sz_) && aligned(dz, v * sz_)));
    a.wide = vec && C % (16 / sx_) == 0 && rows_vec(x, sx_, B, T, a.xbs, a.xts, 16) &&
             rows_vec(dy, sx_, B, T, a.dybs, a.dyts, 16) && (a.zhead || rows_vec(z, sz_, B, T, a.zbs, a.zts, 16));
    use_unit(kGatedBwdUnit, x_dtype);
    return with_x(x_dtype, [&](auto t) {
        return gated::launch_bwd<decltype(t)>(a, gated_form(gate, write, tau), vec, static_cast<cudaStream_t>(stream));
    });
}

lattice_status lattice_gated_step(const float* h, float* h_out, const void* x, lattice_dtype x_dtype,
                                  long long x_batch_stride, const void* z, lattice_dtype z_dtype,
                                  long long z_batch_stride, int z_per_head, void* y, int B, int H, int d,
                                  lattice_gate gate, lattice_write write, float tau, void* stream) {
    lattice_status s = check_gated(x_dtype, z_dtype, z_per_head, B, 1, H, d, gate, write, tau);
    if (s != LATTICE_OK) return s;
    const long long C = (long long)H * d, Cz = z_per_head ? H : C;
    const size_t sx_ = type_size(x_dtype), sz_ = type_size(z_dtype);
    if (!h || !h_out || !x || !z || !y) return LATTICE_ERR_INVALID_ARG;
    Span sx, sz;
    if (!strided_span(x, sx_, B, 1, C, x_batch_stride, 0, &sx) || !strided_span(z, sz_, B, 1, Cz, z_batch_stride, 0, &sz))
        return LATTICE_ERR_INVALID_ARG;
    if (!aligned(h, 4) || !aligned(h_out, 4) || !aligned(x, sx_) || !aligned(z, sz_) || !aligned(y, sx_))
        return LATTICE_ERR_INVALID_ARG;
    const size_t nh = (size_t)B * C * 4;
    const Span ins[] = {sx, sz, span(h, nh)}, outs[] = {span(h_out, nh), span(y, (size_t)B * C * sx_)};
    if (clash(ins, 3, outs, 2, h, h_out)) return LATTICE_ERR_INVALID_ARG;
    GatedArgs a = {};
    a.x = x; a.z = z; a.h0 = h; a.h_out = h_out; a.y = y;
    a.xbs = x_batch_stride; a.zbs = z_batch_stride;
    a.B = B; a.T = 1; a.C = (int)C; a.d = d; a.tau = tau;
    a.z32 = z_dtype == LATTICE_F32; a.zhead = z_per_head != 0;
    if (gate == LATTICE_GATE_LOGIT && tau != 1.f) gated_poly(a);
    const bool vec = gated_vec(a, sx_, kStepVec) && rows_vec(x, sx_, B, 1, a.xbs, 0, kStepVec * sx_) &&
                     (a.zhead || rows_vec(z, sz_, B, 1, a.zbs, 0, kStepVec * sz_));
    return with_x(x_dtype, [&](auto t) {
        return gated::launch_step<decltype(t)>(a, gated_form(gate, write, tau), vec, static_cast<cudaStream_t>(stream));
    });
}

lattice_status lattice_block_norm_fwd(const void* y, lattice_dtype y_dtype, long long y_stride, const void* gate,
                                      long long gate_stride, const void* residual, lattice_dtype residual_dtype,
                                      long long residual_stride, const void* w_post, const void* w_pre,
                                      lattice_dtype w_dtype, void* r_out, void* n_out, lattice_dtype dtype, long long N,
                                      int G, int D, lattice_act act, int post_norm, float scale, float eps, void* stream) {
    if (!residual) residual_dtype = dtype;
    NormArgs a;
    lattice_status s = check_norm(a, y, y_dtype, y_stride, gate, gate_stride, residual, residual_dtype, residual_stride, w_post,
                                  w_pre, w_dtype, dtype, N, G, D, act, post_norm, scale, eps);
    if (s != LATTICE_OK) return s;
    if ((N > 0 && !r_out) || (N > 0 && w_pre && !n_out) || !aligned(r_out, type_size(residual_dtype)) || !aligned(n_out, type_size(dtype)))
        return LATTICE_ERR_INVALID_ARG;
    if (N == 0) return LATTICE_OK;
    const size_t n = (size_t)N * D;
    Span sy, sg = {}, sr = {};
    if (!group_span(y, y_dtype, N, G, D, y_stride, &sy) || !group_span(gate, dtype, N, G, D, gate_stride, &sg) ||
        !group_span(residual, residual_dtype, N, G, D, residual_stride, &sr))
        return LATTICE_ERR_INVALID_ARG;
    if (!gate) sg = Span{};
    if (!residual) sr = Span{};
    const size_t wb = (size_t)D * type_size(w_dtype);
    const Span ins[] = {sy, sg, sr, span(w_post, w_post ? wb : 0), span(w_pre, w_pre ? wb : 0)};
    const Span outs[] = {span(r_out, n * type_size(residual_dtype)), span(n_out, n_out ? n * type_size(dtype) : 0)};
    if (clash(ins, 5, outs, 2, residual, r_out)) return LATTICE_ERR_INVALID_ARG;
    a.r_out = r_out; a.n_out = n_out;
    a.r32 = residual_dtype == LATTICE_F32;
    const bool vec = D % 8 == 0 && norm_rows_vec(y, y_dtype, N, G, y_stride) && norm_rows_vec(gate, dtype, N, G, gate_stride) &&
                     norm_rows_vec(residual, residual_dtype, N, G, residual_stride) && aligned(w_post, 16) &&
                     aligned(w_pre, 16) && aligned(r_out, 16) && aligned(n_out, 16);
    const bool shift = D % 8 != 0 && D + 7 <= kNormMaxD && norm_rows_shift(y, y_dtype, N, G, D, y_stride) &&
                       norm_rows_shift(gate, dtype, N, G, D, gate_stride) &&
                       norm_rows_shift(residual, residual_dtype, N, G, D, residual_stride) && aligned(r_out, 16) &&
                       aligned(n_out, 16);
    const int mode = vec ? kNormVec : shift ? kNormShift : kNormOdd;
    use_unit(kNormUnit, dtype);
    return with_x(dtype, [&](auto t) {
        return norm::launch_norm<decltype(t)>(false, a, mode, nullptr, static_cast<cudaStream_t>(stream));
    });
}

size_t lattice_block_norm_bwd_workspace_bytes(long long N, int D) {
    if (N < 0 || N > 0x7fffffffLL || D < 1 || D > kNormMaxD) return 0;
    return (size_t)norm_parts(N, D) * 2 * D * 4;
}

lattice_status lattice_block_norm_bwd(const void* y, lattice_dtype y_dtype, long long y_stride, const void* gate,
                                      long long gate_stride, const void* residual, lattice_dtype residual_dtype,
                                      long long residual_stride, const void* w_post, const void* w_pre,
                                      lattice_dtype w_dtype, const void* dr, lattice_dtype dr_dtype, long long dr_stride,
                                      const void* dn, long long dn_stride, void* dy, void* dgate, void* dresidual,
                                      float* dw_post, float* dw_pre, void* workspace, size_t workspace_bytes,
                                      lattice_dtype dtype, long long N, int G, int D, lattice_act act, int post_norm,
                                      float scale, float eps, void* stream) {
    if (!residual) residual_dtype = dtype;
    if (!dr) dr_dtype = residual_dtype;
    NormArgs a;
    lattice_status s = check_norm(a, y, y_dtype, y_stride, gate, gate_stride, residual, residual_dtype, residual_stride, w_post,
                                  w_pre, w_dtype, dtype, N, G, D, act, post_norm, scale, eps);
    if (s != LATTICE_OK) return s;
    if (!type_ok(dr_dtype) || dr_stride < 0 || dn_stride < 0) return LATTICE_ERR_INVALID_ARG;
    if ((dr_dtype != LATTICE_F32 && dr_dtype != dtype) || dr_stride > kNormMaxStride || dn_stride > kNormMaxStride)
        return LATTICE_ERR_UNSUPPORTED;
    if (residual && dr && dr_dtype != residual_dtype) return LATTICE_ERR_UNSUPPORTED;
    if (N > 0 && ((!dr && !dn) || !dy || (gate && !dgate) || (residual && !dresidual))) return LATTICE_ERR_INVALID_ARG;
    if ((!gate && dgate) || (!residual && dresidual) || (w_pre && N > 0 && !dn) || (dw_post && !w_post) || (dw_pre && !w_pre))
        return LATTICE_ERR_INVALID_ARG;
    const bool dw = dw_post || dw_pre;
    const size_t need = dw ? lattice_block_norm_bwd_workspace_bytes(N, D) : 0;
    if (need && (!workspace || workspace_bytes < need)) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(dr, type_size(dr_dtype)) || !aligned(dn, type_size(dtype)) || !aligned(dy, type_size(y_dtype)) ||
        !aligned(dgate, type_size(dtype)) || !aligned(dresidual, type_size(residual_dtype)) || !aligned(dw_post, 4) ||
        !aligned(dw_pre, 4) || (need && !aligned(workspace, 16)))
        return LATTICE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        for (float* w : {dw_post, dw_pre}) {
            cudaError_t e = w ? cudaMemsetAsync(w, 0, (size_t)D * 4, st) : cudaSuccess;
            if (e != cudaSuccess) return cuda_fail(e);
        }
        return LATTICE_OK;
    }
    const size_t n = (size_t)N * D;
    Span sy, sg = {}, sr = {}, sdr = {}, sdn = {};
    if (!group_span(y, y_dtype, N, G, D, y_stride, &sy) || !group_span(gate, dtype, N, G, D, gate_stride, &sg) ||
        !group_span(residual, residual_dtype, N, G, D, residual_stride, &sr) ||
        !group_span(dr, dr_dtype, N, G, D, dr_stride, &sdr) || !group_span(dn, dtype, N, G, D, dn_stride, &sdn))
        return LATTICE_ERR_INVALID_ARG;
    if (!gate) sg = Span{};
    if (!residual) sr = Span{};
    if (!dr) sdr = Span{};
    if (!dn) sdn = Span{};
    const size_t wb = (size_t)D * type_size(w_dtype);
    const Span ins[] = {sy, sg, sr, sdr, sdn, span(w_post, w_post ? wb : 0), span(w_pre, w_pre ? wb : 0)};
    const Span outs[] = {span(dy, n * type_size(y_dtype)), span(dgate, dgate ? n * type_size(dtype) : 0),
                         span(dresidual, dresidual ? n * type_size(residual_dtype) : 0),
                         span(dw_post, dw_post ? (size_t)D * 4 : 0), span(dw_pre, dw_pre ? (size_t)D * 4 : 0),
                         span(workspace, need)};
    if (clash(ins, 7, outs, 6, nullptr, nullptr)) return LATTICE_ERR_INVALID_ARG;
    a.dr = dr; a.dn = dn; a.dy = dy; a.dgate = dgate; a.dresidual = dresidual;
    a.parts = dw ? static_cast<float*>(workspace) : nullptr;
    a.drs = (unsigned)dr_stride; a.dns = (unsigned)dn_stride;
    a.r32 = (residual ? residual_dtype : dr_dtype) == LATTICE_F32;
    const bool vec = D % 8 == 0 && norm_rows_vec(y, y_dtype, N, G, y_stride) && norm_rows_vec(gate, dtype, N, G, gate_stride) &&
                     norm_rows_vec(residual, residual_dtype, N, G, residual_stride) &&
                     norm_rows_vec(dr, dr_dtype, N, G, dr_stride) && norm_rows_vec(dn, dtype, N, G, dn_stride) &&
                     aligned(w_post, 16) && aligned(w_pre, 16) && aligned(dy, 16) && aligned(dgate, 16) &&
                     aligned(dresidual, 16);
    const bool shift = D % 8 != 0 && D + 7 <= kNormMaxD && norm_rows_shift(y, y_dtype, N, G, D, y_stride) &&
                       norm_rows_shift(gate, dtype, N, G, D, gate_stride) &&
                       norm_rows_shift(residual, residual_dtype, N, G, D, residual_stride) &&
                       norm_rows_shift(dr, dr_dtype, N, G, D, dr_stride) && norm_rows_shift(dn, dtype, N, G, D, dn_stride) &&
                       aligned(dy, 16) && aligned(dgate, 16) && aligned(dresidual, 16);
    const int mode = vec ? kNormVec : shift ? kNormShift : kNormOdd;
    int groups = 0;
    use_unit(kNormUnit, dtype);
    s = with_x(dtype, [&](auto t) { return norm::launch_norm<decltype(t)>(true, a, mode, &groups, st); });
    return s != LATTICE_OK || !dw ? s : launch_norm_dw(a, groups, dw_post, dw_pre, st);
}

lattice_status lattice_short_conv_fwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride, long long x_token_stride,
                                      const void* w, const void* bias, lattice_dtype w_dtype, const void* state, void* state_out,
                                      void* y, const int* lengths, int B, int T, int C, int K, lattice_act act, void* stream) {
    lattice_status s = check_conv(x_dtype, w_dtype, B, T, C, K, act);
    if (s != LATTICE_OK) return s;
    const size_t sx = type_size(x_dtype), sw = type_size(w_dtype), sb = (size_t)B * (K - 1) * C * sx;
    Span xs;
    if (!strided_span(x, sx, B, T, C, x_batch_stride, x_token_stride, &xs)) return LATTICE_ERR_INVALID_ARG;
    if (!w || (T > 0 && (!x || !y))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(x, sx) || !aligned(y, sx) || !aligned(state, sx) || !aligned(state_out, sx) || !aligned(w, sw) || !aligned(bias, sw) ||
        !aligned(lengths, 4))
        return LATTICE_ERR_INVALID_ARG;
    const Span ins[] = {xs, span(w, (size_t)C * K * sw), span(bias, bias ? (size_t)C * sw : 0), span(state, state ? sb : 0),
                        span(lengths, lengths ? (size_t)B * 4 : 0)};
    const Span outs[] = {span(y, (size_t)B * T * C * sx), span(state_out, state_out ? sb : 0)};
    if (clash(ins, 5, outs, 2, state, state_out)) return LATTICE_ERR_INVALID_ARG;
    ConvArgs a;
    conv_args(a, x, x_dtype, x_batch_stride, x_token_stride, w, bias, w_dtype, state, lengths, B, T, C, K, act);
    a.y = y;
    a.state_out = K > 1 ? state_out : nullptr;
    const int V = conv_width(a, sx, sw);
    a.run = conv_run(B, T, C, K, false, V);
    a.runs = T > a.run ? (int)((T + (long long)a.run - 1) / a.run) : 1;
    return with_x(x_dtype, [&](auto t) { return conv::launch<decltype(t)>(a, kConvFwd, V, static_cast<cudaStream_t>(stream)); });
}

size_t lattice_short_conv_bwd_workspace_bytes(int B, int T, int C, int K) {
    if (check_conv(LATTICE_F32, LATTICE_F32, B, T, C, K, LATTICE_ACT_NONE) != LATTICE_OK) return 0;
    return conv_workspace(B, T > 0 ? T : 1, C, K);
}

lattice_status lattice_short_conv_bwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride, long long x_token_stride,
                                      const void* w, const void* bias, lattice_dtype w_dtype, const void* state, const void* dy,
                                      long long dy_batch_stride, long long dy_token_stride, const void* dstate_out, void* dx,
                                      float* dw, float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                                      const int* lengths, int B, int T, int C, int K, lattice_act act, void* stream) {
    lattice_status s = check_conv(x_dtype, w_dtype, B, T, C, K, act);
    if (s != LATTICE_OK) return s;
    const size_t sx = type_size(x_dtype), sw = type_size(w_dtype), sb = (size_t)B * (K - 1) * C * sx;
    Span xs, ys;
    if (!strided_span(x, sx, B, T, C, x_batch_stride, x_token_stride, &xs) ||
        !strided_span(dy, sx, B, T, C, dy_batch_stride, dy_token_stride, &ys))
        return LATTICE_ERR_INVALID_ARG;
    if (!w || (T > 0 && (!x || !dy || !dx)) || (dbias && !bias) || (dstate && !state)) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(x, sx) || !aligned(dy, sx) || !aligned(dx, sx) || !aligned(state, sx) || !aligned(dstate, sx) ||
        !aligned(dstate_out, sx) || !aligned(w, sw) || !aligned(bias, sw) || !aligned(dw, 4) || !aligned(dbias, 4) || !aligned(lengths, 4))
        return LATTICE_ERR_INVALID_ARG;
    const bool sums = dw || dbias;
    const size_t need = sums ? lattice_short_conv_bwd_workspace_bytes(B, T, C, K) : 0;
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return LATTICE_ERR_INVALID_ARG;
    const Span ins[] = {xs, ys, span(w, (size_t)C * K * sw), span(bias, bias ? (size_t)C * sw : 0), span(state, state ? sb : 0),
                        span(dstate_out, dstate_out ? sb : 0), span(lengths, lengths ? (size_t)B * 4 : 0)};
    const Span outs[] = {span(dx, (size_t)B * T * C * sx), span(dw, dw ? (size_t)C * K * 4 : 0), span(dbias, dbias ? (size_t)C * 4 : 0),
                         span(dstate, dstate ? sb : 0), span(workspace, need)};
    if (clash(ins, 7, outs, 5, nullptr, nullptr)) return LATTICE_ERR_INVALID_ARG;
    ConvArgs a;
    conv_args(a, x, x_dtype, x_batch_stride, x_token_stride, w, bias, w_dtype, state, lengths, B, T, C, K, act);
    a.dy = dy; a.ybs = dy_batch_stride; a.yts = dy_token_stride;
    a.dx = dx; a.dw = dw; a.dbias = dbias;
    a.dstate = K > 1 ? dstate : nullptr;
    a.dstate_out = K > 1 ? dstate_out : nullptr;
    a.parts = sums ? static_cast<float*>(workspace) : nullptr;
    const int V = conv_width(a, sx, sw);
    a.run = conv_run(B, T, C, K, true, V);
    a.runs = T > a.run ? (int)((T + (long long)a.run - 1) / a.run) : 1;
    return with_x(x_dtype, [&](auto t) { return conv::launch<decltype(t)>(a, kConvBwd, V, static_cast<cudaStream_t>(stream)); });
}

lattice_status lattice_short_conv_step(const void* state, void* state_out, const void* x, lattice_dtype x_dtype,
                                       long long x_batch_stride, const void* w, const void* bias, lattice_dtype w_dtype, void* y,
                                       int B, int C, int K, lattice_act act, void* stream) {
    lattice_status s = check_conv(x_dtype, w_dtype, B, 1, C, K, act);
    if (s != LATTICE_OK) return s;
    const size_t sx = type_size(x_dtype), sw = type_size(w_dtype), sb = (size_t)B * (K - 1) * C * sx;
    Span xs;
    if (!strided_span(x, sx, B, 1, C, x_batch_stride, 0, &xs)) return LATTICE_ERR_INVALID_ARG;
    if (!x || !w || !y || (K > 1 && (!state || !state_out))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(x, sx) || !aligned(y, sx) || !aligned(state, sx) || !aligned(state_out, sx) || !aligned(w, sw) || !aligned(bias, sw))
        return LATTICE_ERR_INVALID_ARG;
    const Span ins[] = {xs, span(w, (size_t)C * K * sw), span(bias, bias ? (size_t)C * sw : 0), span(state, sb)};
    const Span outs[] = {span(y, (size_t)B * C * sx), span(state_out, sb)};
    if (clash(ins, 4, outs, 2, state, state_out)) return LATTICE_ERR_INVALID_ARG;
    ConvArgs a;
    conv_args(a, x, x_dtype, x_batch_stride, 0, w, bias, w_dtype, state, nullptr, B, 1, C, K, act);
    a.y = y; a.state_out = state_out;
    a.run = 8, a.runs = 1;
    const int V = conv_width(a, sx, sw);
    return with_x(x_dtype, [&](auto t) { return conv::launch<decltype(t)>(a, kConvStep, V, static_cast<cudaStream_t>(stream)); });
}

size_t lattice_selective_scan_marks_bytes(int B, int T, int E, int N) {
    if (check_selective(LATTICE_F32, LATTICE_F32, B, T, E, N, 1) != LATTICE_OK) return 0;
    return (size_t)B * ((T + (size_t)kSelMark - 1) / kSelMark) * E * N * 4;
}

size_t lattice_selective_scan_workspace_bytes(int B, int T, int E, int N, int G, int backward) {
    if (check_selective(LATTICE_F32, LATTICE_F32, B, T, E, N, G) != LATTICE_OK) return 0;
    return sel_space(sel_plan(B, T, E, N, G, backward != 0), B, T, E, N, G, backward != 0).bytes();
}

lattice_status lattice_selective_scan_fwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride, long long x_token_stride,
                                          const void* dt, lattice_dtype dt_dtype, long long dt_batch_stride, long long dt_token_stride,
                                          const float* A, const void* b, long long b_batch_stride, long long b_token_stride,
                                          const void* c, long long c_batch_stride, long long c_token_stride, const float* skip,
                                          const void* z, long long z_batch_stride, long long z_token_stride, const float* dt_bias,
                                          int softplus, const float* h0, float* h_out, void* y, float* marks, const int* lengths,
                                          void* workspace, size_t workspace_bytes, int B, int T, int E, int N, int G, void* stream) {
    lattice_status s = check_selective(x_dtype, dt_dtype, B, T, E, N, G);
    if (s != LATTICE_OK) return s;
    SelArgs a;
    SelInputs in;
    s = sel_inputs(a, in, x, x_dtype, x_batch_stride, x_token_stride, dt, dt_dtype, dt_batch_stride, dt_token_stride, A, b,
                   b_batch_stride, b_token_stride, c, c_batch_stride, c_token_stride, skip, z, z_batch_stride, z_token_stride, dt_bias,
                   softplus, lengths, B, T, E, N, G);
    if (s != LATTICE_OK) return s;
    if (T > 0 && !y && !marks) return LATTICE_ERR_INVALID_ARG;
    const size_t sx = type_size(x_dtype), nh = (size_t)B * E * N * 4;
    const SelPlan plan = sel_plan(B, T, E, N, G, false);
    const SelSpace space = sel_space(plan, B, T, E, N, G, false);
    const size_t need = space.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(h0, 4) || !aligned(h_out, 4) || !aligned(y, sx) || !aligned(marks, 16)) return LATTICE_ERR_INVALID_ARG;
    in.s[in.n++] = span(h0, h0 ? nh : 0);
    const Span outs[] = {span(h_out, h_out ? nh : 0), span(y, y ? (size_t)B * T * E * sx : 0),
                         span(marks, marks ? lattice_selective_scan_marks_bytes(B, T, E, N) : 0), span(workspace, need)};
    if (clash(in.s, in.n, outs, 4, h0, h_out)) return LATTICE_ERR_INVALID_ARG;
    a.h0 = h0; a.h_out = h_out; a.y = y; a.marks = marks;
    a.vec = sel_vec(a, sx, sel_width(sel_padded(N) / plan.S));
    a.vec_n = a.vec_n && aligned(h0, 16) && aligned(h_out, 16);
    sel_place(a, plan, space, workspace);
    return with_x(x_dtype, [&](auto t) { return selective::launch_fwd<decltype(t)>(a, plan.S, plan.W, static_cast<cudaStream_t>(stream)); });
}

lattice_status lattice_selective_scan_bwd(const void* x, lattice_dtype x_dtype, long long x_batch_stride, long long x_token_stride,
                                          const void* dt, lattice_dtype dt_dtype, long long dt_batch_stride, long long dt_token_stride,
                                          const float* A, const void* b, long long b_batch_stride, long long b_token_stride,
                                          const void* c, long long c_batch_stride, long long c_token_stride, const float* skip,
                                          const void* z, long long z_batch_stride, long long z_token_stride, const float* dt_bias,
                                          int softplus, const void* dy, long long dy_batch_stride, long long dy_token_stride,
                                          const float* marks, const float* dh_T, void* dx, void* ddt, float* dA, void* db, void* dc,
                                          float* dskip, void* dz, float* ddt_bias, float* dh0, const int* lengths, void* workspace,
                                          size_t workspace_bytes, int B, int T, int E, int N, int G, void* stream) {
    lattice_status s = check_selective(x_dtype, dt_dtype, B, T, E, N, G);
    if (s != LATTICE_OK) return s;
    SelArgs a;
    SelInputs in;
    s = sel_inputs(a, in, x, x_dtype, x_batch_stride, x_token_stride, dt, dt_dtype, dt_batch_stride, dt_token_stride, A, b,
                   b_batch_stride, b_token_stride, c, c_batch_stride, c_token_stride, skip, z, z_batch_stride, z_token_stride, dt_bias,
                   softplus, lengths, B, T, E, N, G);
    if (s != LATTICE_OK) return s;
    if (T > 0 && (!dy || !marks || !dx || !ddt || !db || !dc || (z && !dz))) return LATTICE_ERR_INVALID_ARG;
    if (!dA || !dh0 || (!z && dz) || (dskip && !skip) || (ddt_bias && !dt_bias)) return LATTICE_ERR_INVALID_ARG;
    const size_t sx = type_size(x_dtype), sd = type_size(dt_dtype), nh = (size_t)B * E * N * 4, nt = (size_t)B * T;
    const SelPlan plan = sel_plan(B, T, E, N, G, true);
    const SelSpace space = sel_space(plan, B, T, E, N, G, true);
    const size_t need = space.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return LATTICE_ERR_INVALID_ARG;
    for (const void* p : {dy, (const void*)dx, (const void*)db, (const void*)dc, (const void*)dz})
        if (!aligned(p, sx)) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(ddt, sd) || !aligned(marks, 16) || !aligned(dh_T, 4) || !aligned(dA, 4) || !aligned(dskip, 4) || !aligned(ddt_bias, 4) ||
        !aligned(dh0, 4))
        return LATTICE_ERR_INVALID_ARG;
    Span ys;
    if (!strided_span(dy, sx, B, T, E, dy_batch_stride, dy_token_stride, &ys)) return LATTICE_ERR_INVALID_ARG;
    const Span more[] = {ys, span(marks, lattice_selective_scan_marks_bytes(B, T, E, N)), span(dh_T, dh_T ? nh : 0)};
    const Span outs[] = {span(dx, nt * E * sx), span(ddt, nt * E * sd), span(dz, dz ? nt * E * sx : 0), span(db, nt * G * N * sx),
                         span(dc, nt * G * N * sx), span(dA, (size_t)E * N * 4), span(dskip, dskip ? (size_t)E * 4 : 0),
                         span(ddt_bias, ddt_bias ? (size_t)E * 4 : 0), span(dh0, nh), span(workspace, need)};
    if (clash(in.s, in.n, outs, 10, nullptr, nullptr) || clash(more, 3, outs, 10, nullptr, nullptr)) return LATTICE_ERR_INVALID_ARG;
    a.dy = dy; a.ybs = dy_batch_stride; a.yts = dy_token_stride;
    a.marks = const_cast<float*>(marks); a.dh_T = dh_T;
    a.dx = dx; a.ddt = ddt; a.dz = dz; a.dh0 = dh0; a.db = db; a.dc = dc; a.dA = dA; a.dskip = dskip; a.ddt_bias = ddt_bias;
    a.vec = sel_vec(a, sx, sel_width(sel_padded(N) / 4));
    a.vec_n = a.vec_n && aligned(dh_T, 16) && aligned(dh0, 16);
    sel_place(a, plan, space, workspace);
    return with_x(x_dtype, [&](auto t) { return selective::launch_bwd<decltype(t)>(a, plan.W, static_cast<cudaStream_t>(stream)); });
}

lattice_status lattice_selective_step(const float* h, float* h_out, const void* x, lattice_dtype x_dtype, long long x_batch_stride,
                                      const void* dt, lattice_dtype dt_dtype, long long dt_batch_stride, const float* A, const void* b,
                                      long long b_batch_stride, const void* c, long long c_batch_stride, const float* skip,
                                      const void* z, long long z_batch_stride, const float* dt_bias, int softplus, void* y, int B,
                                      int E, int N, int G, void* stream) {
    lattice_status s = check_selective(x_dtype, dt_dtype, B, 1, E, N, G);
    if (s != LATTICE_OK) return s;
    SelArgs a;
    SelInputs in;
    s = sel_inputs(a, in, x, x_dtype, x_batch_stride, 0, dt, dt_dtype, dt_batch_stride, 0, A, b, b_batch_stride, 0, c, c_batch_stride, 0,
                   skip, z, z_batch_stride, 0, dt_bias, softplus, nullptr, B, 1, E, N, G);
    if (s != LATTICE_OK) return s;
    const size_t sx = type_size(x_dtype), nh = (size_t)B * E * N * 4;
    if (!h || !h_out || !y || !aligned(h, 4) || !aligned(h_out, 4) || !aligned(y, sx)) return LATTICE_ERR_INVALID_ARG;
    in.s[in.n++] = span(h, nh);
    const Span outs[] = {span(h_out, nh), span(y, (size_t)B * E * sx)};
    if (clash(in.s, in.n, outs, 2, h, h_out)) return LATTICE_ERR_INVALID_ARG;
    a.h0 = h; a.h_out = h_out; a.y = y;
    a.vec_n = a.vec_n && aligned(h, 16) && aligned(h_out, 16);
    a.vec = a.vec_n && rows_vec(b, sx, B, 1, b_batch_stride, 0, 4 * sx) && rows_vec(c, sx, B, 1, c_batch_stride, 0, 4 * sx);
    return with_x(x_dtype, [&](auto t) { return selective::launch_step<decltype(t)>(a, static_cast<cudaStream_t>(stream)); });
}

lattice_status lattice_layer_norm_fwd(const void* x, lattice_dtype x_dtype, long long x_stride, const void* residual,
                                      lattice_dtype residual_dtype, long long residual_stride, const void* w, const void* b,
                                      lattice_dtype w_dtype, void* r_out, void* n_out, lattice_dtype dtype, long long N, int G, int D,
                                      float eps, void* stream) {
    if (!residual) residual_dtype = x_dtype;
    NormArgs a;
    lattice_status s = check_norm(a, x, x_dtype, x_stride, nullptr, 0, residual, residual_dtype, residual_stride, w, b, w_dtype, dtype,
                                  N, G, D, LATTICE_ACT_NONE, 1, 1.f, eps);
    if (s != LATTICE_OK) return s;
    if ((N > 0 && (!n_out || (residual && !r_out))) || (!residual && r_out) || !aligned(r_out, type_size(residual_dtype)) ||
        !aligned(n_out, type_size(dtype)))
        return LATTICE_ERR_INVALID_ARG;
    if (N == 0) return LATTICE_OK;
    const size_t n = (size_t)N * D, wb = (size_t)D * type_size(w_dtype);
    Span sx, sr = {};
    if (!group_span(x, x_dtype, N, G, D, x_stride, &sx) || !group_span(residual, residual_dtype, N, G, D, residual_stride, &sr))
        return LATTICE_ERR_INVALID_ARG;
    if (!residual) sr = Span{};
    const Span ins[] = {sx, sr, span(w, w ? wb : 0), span(b, b ? wb : 0)};
    const Span outs[] = {span(r_out, r_out ? n * type_size(residual_dtype) : 0), span(n_out, n * type_size(dtype))};
    if (clash(ins, 4, outs, 2, residual, r_out)) return LATTICE_ERR_INVALID_ARG;
    a.r_out = r_out; a.n_out = n_out;
    const bool vec = D % 8 == 0 && norm_rows_vec(x, x_dtype, N, G, x_stride) && norm_rows_vec(residual, residual_dtype, N, G, residual_stride) &&
                     aligned(r_out, 16) && aligned(n_out, 16);
    const bool shift = D % 8 != 0 && D + 7 <= kNormMaxD && norm_rows_shift(x, x_dtype, N, G, D, x_stride) &&
                       norm_rows_shift(residual, residual_dtype, N, G, D, residual_stride) && aligned(r_out, 16) && aligned(n_out, 16);
    use_unit(kLayerNormUnit, dtype);
    return with_x(dtype, [&](auto t) {
        return norm::launch_layer<decltype(t)>(false, a, vec ? kNormVec : shift ? kNormShift : kNormOdd, nullptr, static_cast<cudaStream_t>(stream));
    });
}

size_t lattice_layer_norm_bwd_workspace_bytes(long long N, int D) {
    if (N < 0 || N > 0x7fffffffLL || D < 1 || D > kNormMaxD) return 0;
    return (size_t)layer_parts(N, D) * 2 * D * 4;
}

lattice_status lattice_layer_norm_bwd(const void* r, lattice_dtype r_dtype, long long r_stride, const void* dn, long long dn_stride,
                                      const void* dr, long long dr_stride, const void* w, lattice_dtype w_dtype, void* dr_out, void* dx,
                                      lattice_dtype x_dtype, float* dw, float* db, void* workspace, size_t workspace_bytes,
                                      lattice_dtype dtype, long long N, int G, int D, float eps, void* stream) {
    if (!dx) x_dtype = r_dtype;
    NormArgs a;
    lattice_status s = check_norm(a, r, r_dtype, r_stride, nullptr, 0, nullptr, r_dtype, 0, w, nullptr, w_dtype, dtype, N, G, D,
                                  LATTICE_ACT_NONE, 1, 1.f, eps);
    if (s != LATTICE_OK) return s;
    if (!type_ok(x_dtype) || dn_stride < 0 || dr_stride < 0) return LATTICE_ERR_INVALID_ARG;
    if ((x_dtype != LATTICE_F32 && x_dtype != dtype) || dn_stride > kNormMaxStride || dr_stride > kNormMaxStride) return LATTICE_ERR_UNSUPPORTED;
    if ((N > 0 && (!dn || !dr_out)) || (dw && !w)) return LATTICE_ERR_INVALID_ARG;
    const bool sums = dw || db;
    const size_t need = sums ? lattice_layer_norm_bwd_workspace_bytes(N, D) : 0;
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return LATTICE_ERR_INVALID_ARG;
    if (!aligned(dn, type_size(dtype)) || !aligned(dr, type_size(r_dtype)) || !aligned(dr_out, type_size(r_dtype)) ||
        !aligned(dx, type_size(x_dtype)) || !aligned(dw, 4) || !aligned(db, 4))
        return LATTICE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        for (float* p : {dw, db}) {
            cudaError_t e = p ? cudaMemsetAsync(p, 0, (size_t)D * 4, st) : cudaSuccess;
            if (e != cudaSuccess) return cuda_fail(e);
        }
        return LATTICE_OK;
    }
    const size_t n = (size_t)N * D;
    Span sr, sdn, sdr = {};
    if (!group_span(r, r_dtype, N, G, D, r_stride, &sr) || !group_span(dn, dtype, N, G, D, dn_stride, &sdn) ||
        !group_span(dr, r_dtype, N, G, D, dr_stride, &sdr))
        return LATTICE_ERR_INVALID_ARG;
    if (!dr) sdr = Span{};
    const Span ins[] = {sr, sdn, sdr, span(w, w ? (size_t)D * type_size(w_dtype) : 0)};
    const Span outs[] = {span(dr_out, n * type_size(r_dtype)), span(dx, dx ? n * type_size(x_dtype) : 0),
                         span(dw, dw ? (size_t)D * 4 : 0), span(db, db ? (size_t)D * 4 : 0), span(workspace, need)};
    if (clash(ins, 4, outs, 5, nullptr, nullptr)) return LATTICE_ERR_INVALID_ARG;
    a.dn = dn; a.dr = dr; a.dresidual = dr_out; a.dy = dx;
    a.dns = (unsigned)dn_stride; a.drs = (unsigned)dr_stride;
    a.parts = sums ? static_cast<float*>(workspace) : nullptr;
    a.r32 = r_dtype == LATTICE_F32; a.y32 = x_dtype == LATTICE_F32;
    const bool vec = D % 8 == 0 && norm_rows_vec(r, r_dtype, N, G, r_stride) && norm_rows_vec(dn, dtype, N, G, dn_stride) &&
                     norm_rows_vec(dr, r_dtype, N, G, dr_stride) && aligned(dr_out, 16) && aligned(dx, 16);
    const bool shift = D % 8 != 0 && D + 7 <= kNormMaxD && norm_rows_shift(r, r_dtype, N, G, D, r_stride) &&
                       norm_rows_shift(dn, dtype, N, G, D, dn_stride) && norm_rows_shift(dr, r_dtype, N, G, D, dr_stride) &&
                       aligned(dr_out, 16) && aligned(dx, 16);
    int groups = 0;
    use_unit(kLayerNormUnit, dtype);
    s = with_x(dtype, [&](auto t) {
        return norm::launch_layer<decltype(t)>(true, a, vec ? kNormVec : shift ? kNormShift : kNormOdd, &groups, st);
    });
    return s != LATTICE_OK || !sums ? s : launch_norm_dw(a, groups, dw, db, st);
}

lattice_status lattice_selftest_bounded_wait(unsigned long long limit_ns, void* stream) {
    if (limit_ns < 1 || limit_ns > 1000000000ull) return LATTICE_ERR_INVALID_ARG;
    bounded_wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns);
    return launch_status();
}

lattice_status lattice_get_device_status(void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e);
    // every translation unit's copy of the status word (each unit is a module of its own), the layer
    // operators' where they have been used (their one-token form has no waits)
    const struct {
        cudaError_t (*read)(unsigned int*);
        bool used;
    } units[] = {{read_clear_module_status, true},
                 {status_simt_exact, true},
                 {status_simt_chunked, true},
                 {status_step, true},
                 {status_bwd, true},
                 {status_tc, true},
                 {status_norm_f32, unit_used(kNormUnit, LATTICE_F32)},
                 {status_norm_bf16, unit_used(kNormUnit, LATTICE_BF16)},
                 {status_norm_f16, unit_used(kNormUnit, LATTICE_F16)},
                 {status_lnorm_f32, unit_used(kLayerNormUnit, LATTICE_F32)},
                 {status_lnorm_bf16, unit_used(kLayerNormUnit, LATTICE_BF16)},
                 {status_lnorm_f16, unit_used(kLayerNormUnit, LATTICE_F16)},
                 {status_gated_fwd_f32, unit_used(kGatedFwdUnit, LATTICE_F32)},
                 {status_gated_fwd_bf16, unit_used(kGatedFwdUnit, LATTICE_BF16)},
                 {status_gated_fwd_f16, unit_used(kGatedFwdUnit, LATTICE_F16)},
                 {status_gated_bwd_f32, unit_used(kGatedBwdUnit, LATTICE_F32)},
                 {status_gated_bwd_bf16, unit_used(kGatedBwdUnit, LATTICE_BF16)},
                 {status_gated_bwd_f16, unit_used(kGatedBwdUnit, LATTICE_F16)}};
    unsigned int any = 0;
    for (const auto& unit : units) {
        if (!unit.used) continue;
        unsigned int v = 0;
        e = unit.read(&v);
        if (e != cudaSuccess) return cuda_fail(e);
        any |= v;
    }
    return any ? LATTICE_ERR_TIMEOUT : LATTICE_OK;
}

const char* lattice_last_cuda_error(void) { return g_last_error; }

}  // extern "C"

// ---- backward pass without allocation: scratch in a static device array
namespace {

constexpr size_t kNoAllocScratchBytes = LATTICE_NOALLOC_SCRATCH_BYTES;
constexpr int kNoAllocCacheEntries = 64;

static __device__ __align__(256) float g_noalloc_scratch[kNoAllocScratchBytes / sizeof(float)];

// The array's device address differs from context to context (each context loads its
// own copy of the module), so the looked-up address is cached per context, keyed by
// the driver's unique context id. A caller running inside its own driver-API context,
// or a process that reset the device and so got a new primary context, gets a fresh
// lookup instead of an address that belongs to another context.
struct NoAllocEntry {
    unsigned long long ctx_id;
    void* addr;
};
std::mutex g_noalloc_mutex;
NoAllocEntry g_noalloc_cache[kNoAllocCacheEntries] = {};
int g_noalloc_next = 0;

typedef CUresult (*PfnCtxGetCurrent)(CUcontext*);
typedef CUresult (*PfnCtxGetId)(CUcontext, unsigned long long*);

// Unique id of the context current on this thread (false if none is current).
bool current_ctx_id(unsigned long long* id) {
    static PfnCtxGetCurrent get_current = nullptr;
    static PfnCtxGetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<PfnCtxGetCurrent>(p);
        p = nullptr;
        if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<PfnCtxGetId>(p);
    });
    CUcontext ctx = nullptr;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx) return false;
    return get_id(ctx, id) == CUDA_SUCCESS;
}

// Device address of g_noalloc_scratch in the current context, looked up once per
// context with cudaGetSymbolAddress (a host-side query, no stream work). In host
// code the array's name is only a host-side stand-in, never a device address.
lattice_status noalloc_scratch(void** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    unsigned long long id = 0;
    bool have_id = current_ctx_id(&id);
    if (have_id) {
        for (const NoAllocEntry& en : g_noalloc_cache)
            if (en.addr && en.ctx_id == id) {
                *out = en.addr;
                return LATTICE_OK;
            }
    }
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);  // makes the device's primary context current if none is
    if (e != cudaSuccess) return cuda_fail(e);
    if (!have_id) have_id = current_ctx_id(&id);
    if (have_id) {
        g_noalloc_cache[g_noalloc_next] = NoAllocEntry{id, p};
        g_noalloc_next = (g_noalloc_next + 1) % kNoAllocCacheEntries;
    }
    *out = p;
    return LATTICE_OK;
}

}  // namespace

extern "C" lattice_status lattice_scan_bwd_noalloc(
    const void* x, lattice_dtype x_dtype, const float* c, const void* q, lattice_dtype q_dtype,
    const float* mu, const float* eta, const float* S0, const float* dy, const float* dS_T,
    float* dx, float* dc, float* dq, float* dmu, float* deta, float* dS0, int B, int T, int H,
    int m, int d, int chunk_size, int seg_tokens, void* stream) {
    const size_t need = lattice_scan_bwd_workspace_bytes(B, T, H, m, d, chunk_size, seg_tokens);
    if (need == 0)  // a rejected shape: lattice_scan_bwd names the error before using the workspace
        return lattice_scan_bwd(x, x_dtype, c, q, q_dtype, mu, eta, S0, dy, dS_T, dx, dc, dq, dmu,
                                deta, dS0, nullptr, 0, B, T, H, m, d, chunk_size, seg_tokens, stream);
    if (need > kNoAllocScratchBytes) return LATTICE_ERR_UNSUPPORTED;
    void* scratch = nullptr;
    lattice_status s = noalloc_scratch(&scratch);
    if (s != LATTICE_OK) return s;
    return lattice_scan_bwd(x, x_dtype, c, q, q_dtype, mu, eta, S0, dy, dS_T, dx, dc, dq, dmu, deta,
                            dS0, scratch, kNoAllocScratchBytes, B, T, H, m, d, chunk_size, seg_tokens,
                            stream);
}

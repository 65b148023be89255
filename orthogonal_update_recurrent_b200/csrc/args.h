// args.h -- kernel argument blocks and the size rules the host needs, with no device
// code, so that the C ABI's translation unit can build them without compiling any
// kernel. Each kernel family's header includes this file.
#pragma once
#include <stddef.h>

#if defined(__CUDACC__)
#define LATTICE_HD __host__ __device__
#else
#define LATTICE_HD
#endif

namespace lattice {

constexpr int kMaxM = 256;  // most slots per head on every path

// scan_simt.cuh, chunk_tc.cuh, chunk_split.cuh, chunk_reg.cuh
struct ScanArgs {
    const void* x; bool x_bf16;
    const float* c;
    const void* q; bool q_bf16;
    const float* mu;
    const float* eta;            // may be null (=> 1)
    const float* S0;
    float* S_out;
    float* y;
    int B, T, H, m, chunk;
    int cnorm;  // chunked CUDA-core path: no per-token normaliser, unit slots after each chunk
    int G;      // SPLIT kernels: CTAs per sequence (a cluster), each owning spc slots
    int spc;
};

// step.cuh: decode step
struct StepArgs {
    float* S;
    const void* x; bool x_bf16;
    const float* c;
    const void* q; bool q_bf16;
    const float* mu;
    const float* eta;  // may be null
    float* y;
    int B, H, m;
};

// step.cuh: read-out of a given state
struct ReadoutArgs {
    const float* S;
    const void* q; bool q_bf16;
    float* y;
    int B, H, m;
};

// scan_bwd.cuh: backward pass
struct BwdArgs {
    const void* x; bool x_bf16;
    const float* c;
    const void* q; bool q_bf16;
    const float* mu;
    const float* eta;  // may be null (=> 1)
    const float* S0;
    const float* dy;
    const float* dST;  // may be null (=> 0)
    float* dx; float* dc; float* dq; float* dmu;
    float* deta;       // may be null
    float* dS0;
    float* ws;         // workspace: per (b,h) and CTA, (nseg - 1) checkpoints then the L-token tape
    int B, T, H, m, chunk, seg;
    int G;             // CTAs per sequence (a cluster when > 1)
    int spc;           // slots per CTA
};

// Floats of backward workspace per (b,h) sequence and CTA (m: the CTA's slots).
LATTICE_HD inline size_t bwd_ws_floats_per_seq(int T, int m, int D, int seg) {
    const int nseg = T > 0 ? (T + seg - 1) / seg : 1;
    return (size_t)(nseg - 1 + seg) * m * D;
}

// Chunk-parallel backward (chunk_bwd.cuh): 16 slots per CTA, 512 threads, chunks of
// 2..64 tokens, a sequence's slots on a cluster of ceil(m/16) <= 8 CTAs.
constexpr int kCbSlots = 16;
constexpr int kCbThreads = 512;
constexpr int kCbMaxL = 64;
constexpr int kCbMaxG = 8;

inline bool chunk_bwd_supported(int m, int d, int chunk) {
    return chunk >= 2 && chunk <= kCbMaxL && (d == 32 || d == 64 || d == 128) && m >= 1 &&
           m <= kCbMaxG * kCbSlots;
}
inline int chunk_bwd_ctas(int m) { return (m + kCbSlots - 1) / kCbSlots; }
// Workspace floats of the chunk-parallel backward: each CTA's slots of every chunk-start state.
inline size_t chunk_bwd_ws_floats(int B, int T, int H, int m, int D, int chunk) {
    const size_t nc = T > 0 ? (size_t)((T + chunk - 1) / chunk) : 0;
    return (size_t)B * H * chunk_bwd_ctas(m) * nc * kCbSlots * D;
}

// gated.cuh: gated linear recurrence
constexpr int kGatedMark = 16;  // tokens between the states the forward pass leaves for the backward pass
constexpr int kGatedMaxK = 16;  // CTAs of a cluster at most

constexpr int kGatedMaxSize = 1 << 30;  // channels, and tokens: tile indices stay within int

constexpr int kGatedPoly = 10;  // coefficients

struct GatedArgs {
    const void* x; const void* z;  // z: fp32 (z32) or x's type, per channel or per head (zhead)
    const float* h0;               // may be null (=> 0)
    float* h_out;                  // forward: may be null
    void* y;                       // forward: may be null
    float* marks;                  // forward: may be null
    const int* lengths;            // may be null (=> T)
    const void* dy; const float* dh_T;
    void* dx; void* dz; float* dh0;
    long long xbs, xts, zbs, zts, dybs, dyts;  // batch and token strides, in elements
    int B, T, C, d;                // C = H*d channels
    int ctiles, K, nmarks;         // channel tiles, CTAs per cluster, marks per sequence
    float tau;
    int squares;                   // tau != 1: poly stands for tau / 2^squares <= 1
    unsigned long long poly[kGatedPoly];  // (1 - (1 + t)^-tau)/t on [0, 1], each coefficient twice
    bool z32, zhead;
    bool wide;                     // rows can be read in 16-byte pieces
    bool zwords;                   // 16-bit gates per head: every token's are whole 32-bit words
};

// block_norm.cuh: norms after and before a block
constexpr int kNormOdd = 0, kNormVec = 1, kNormShift = 2;  // how rows are read
constexpr int kNormMaxD = 16384;
constexpr long long kNormMaxStride = 0x7fffffff;

struct NormArgs {
    const void* y; const void* gate; const void* residual;  // the last two may be null
    const void* w_post; const void* w_pre;                  // may be null (=> 1)
    void* r_out; void* n_out;                               // forward: n_out may be null
    const void* dr; const void* dn;                         // backward: one may be null (=> 0)
    void* dy; void* dgate; void* dresidual;                 // backward: the last two may be null
    float* parts;                                           // backward: weight gradients' sums per CTA, or null
    unsigned ys, gs, rs, drs, dns;                          // between groups of G rows, in elements
    long long N;
    int G, D, tpr, K;                                       // threads per row and CTA, CTAs per row
    int act;
    float scale, eps, inv_d;
    bool post;
    bool y32, r32, w32;                                     // fp32, else the call's type: y; residual, r and dr; weights
};

}  // namespace lattice

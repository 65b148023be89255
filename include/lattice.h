/*
 * lattice.h -- C ABI of the B200 (sm_100a) Lattice compression-layer library.
 *
 * The library computes the state recurrence of "Lattice: Learning to
 * Efficiently Compress the Memory" (Karami, Pascanu, Mirrokni; arXiv
 * 2504.05646) for the similarity objective (h_t = -x_t):
 *
 *   per (batch b, head h), a state of m slots s_i in R^d (rows of S, the
 *   layout of the paper's Appendix D listing), for every token t:
 *     n_i = |s_i|,  p_i = s_i . x_t
 *     w_i = mu_t s_i + eta_t (c_{t,i}/n_i) (x_t - (p_i/n_i^2) s_i)
 *           [§3.1.1 eq. OSR: write only the part of x orthogonal to the slot,
 *            scaled by the writing intensity c; §3.3 eq. dacay_recurrence:
 *            forget gate mu; §3.4 Eq. 14: projection by one dot + one axpy]
 *     s_i <- w_i / |w_i|        [§3.2 eq. normalized_recurrence: unit sphere]
 *     y_t = sum_i q_{t,i} s_i   [read-out with the updated state, §3 General
 *                                Form; Appendix D, y = q @ S_t]
 *   If w_i = 0 (mu = 0 and no orthogonal write) the slot is left unchanged.
 *
 * The chunked form (chunk_size C > 1) is the paper's Eq. 17
 * (recurrence_linear2, §3.4.1 and Appendix B.1): inside a chunk the projection
 * uses the chunk-start state S0 (n_i = |s0_i|, p_i = s0_i . x_t) and the token
 * update is the gated linear recurrence s_i <- g_{t,i} s_i + kappa_{t,i} x_t with
 *   den = mu_t^2 n_i^2 + (eta_t c_{t,i}/n_i)^2 max(0, |x_t|^2 - p_i^2/n_i^2)
 *   g   = n_i (mu_t - eta_t c_{t,i} p_i / n_i^3) / sqrt(den)
 *   kappa = n_i (eta_t c_{t,i} / n_i) / sqrt(den)      [eq. beta_chunk]
 * (g = 1, kappa = 0 where den = 0). The factor n_i = |s0_i| follows the paper's
 * Appendix D listing, whose chunk normaliser keeps each slot's chunk-start
 * norm. Chunks are consecutive blocks of C tokens; the last one may be
 * partial. For unit-norm states, C = 1 is exactly the recurrence above.
 *
 * Layouts (row-major, element strides, no padding):
 *   x    [B][T][H][d]   fp32 or bf16          input written into the slots
 *   c    [B][T][H][m]   fp32                  writing intensities (codes)
 *   q    [B][T][H][m]   fp32 or bf16          read-out queries
 *   mu   [B][T][H]      fp32                  forget gate
 *   eta  [B][T][H]      fp32, or NULL for 1   step size
 *   S    [B][H][m][d]   fp32                  state, one slot per row
 *   y    [B][T][H][d]   fp32                  read-out
 * Decode calls drop the T axis.
 *
 * Ownership and execution: every pointer is caller-owned DEVICE memory. The
 * library allocates nothing and keeps no state that a result depends on besides
 * the device status word (and the static scratch array of
 * lattice_scan_bwd_noalloc, described there). On the host it keeps how many CTAs
 * of a kernel a device holds at once, and which units' status words can be set;
 * a kernel's limit of shared memory is set to the most that its launches take.
 * Every call is asynchronous on `stream` (a cudaStream_t passed as void*,
 * NULL = the legacy default stream) and returns after the launch. Several host
 * threads may call at once, on buffers that no two calls in flight write.
 *
 * Errors: arguments are checked on the host before anything is launched; a
 * failed check launches nothing and returns the code. LATTICE_ERR_CUDA means a
 * launch or attribute call failed (lattice_last_cuda_error has the detail).
 * Device-side waits are bounded: a kernel that gives up sets the status word
 * and returns; lattice_get_device_status() reports it as LATTICE_ERR_TIMEOUT.
 *
 * Supported sizes: d in {16, 32, 64, 128}; 1 <= m <= 256 (m <= 128 for the
 * backward pass); B, H >= 1; T >= 0.
 * The tensor-core chunked kernel serves C = 64, m in {64, 128},
 * d in {64, 128} with bf16 x and q; other chunked shapes run a CUDA-core
 * kernel of the same definition.
 */
#ifndef LATTICE_H_
#define LATTICE_H_

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LATTICE_OK = 0,
    LATTICE_ERR_INVALID_ARG = 1, /* NULL pointer, bad size, partial aliasing  */
    LATTICE_ERR_UNSUPPORTED = 2, /* valid but outside the supported sizes     */
    LATTICE_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed      */
    LATTICE_ERR_TIMEOUT = 4      /* a bounded device-side wait gave up        */
} lattice_status;

/* F16 is accepted by the layer operators only: the gated recurrence, the norms, the short
 * convolution and the selective scan. */
typedef enum { LATTICE_F32 = 0, LATTICE_BF16 = 1, LATTICE_F16 = 2 } lattice_dtype;

/* Objective (§3.1.1, eq. OSR): what each token writes into the slots.
 *   LATTICE_SIM  dot-product similarity objective, h_t = -x_t: slot i takes
 *                the part of x_t orthogonal to it (eq. similarity_recurrence).
 *   LATTICE_DEC  l2 reconstruction objective, h_t = e_t = phi(S) c_t - x_t with
 *                phi(s_i) = s_i/|s_i| (eq. decoding_stateNorm_loss and
 *                eq. decoding_recurrence): slot i takes the part of the
 *                reconstruction residual x_t - sum_j c_tj s_j/|s_j| orthogonal
 *                to it. e is formed from the state the token's projection uses:
 *                the current state (exact recurrence, decode step) or the
 *                chunk-start state (chunked form, as in the Appendix D listing).
 * DEC runs on the CUDA-core kernels only. The tensor-core choices return
 * LATTICE_ERR_UNSUPPORTED for it, and LATTICE_IMPL_AUTO takes the CUDA-core
 * kernel. */
typedef enum { LATTICE_SIM = 0, LATTICE_DEC = 1 } lattice_mode;

/* Kernel choice for chunked scans.
 *   AUTO            picks the fastest kernel that can run the shape (see
 *                   lattice_chunk_impl).
 *   SIMT            the CUDA-core kernel (any chunk size, fp32 or bf16 x/q).
 *   TCGEN05         the tensor-core kernel with one CTA per sequence
 *                   (chunk 64, bf16 x and q, m and d in {64, 128}).
 *   TCGEN05_SPLIT   the tensor-core kernel with each sequence's 64 slots split
 *                   over a cluster of 4 CTAs (chunk 64, bf16 x and q, m = 64,
 *                   d in {64, 128}); for batches with fewer sequences than SMs.
 *   SPLIT_REG       the same split and read-out, with each CTA's share of the
 *                   state held in registers and advanced chunk to chunk by
 *                   warp-synchronous tensor-core MMAs (mma.sync), which keeps the
 *                   per-chunk dependency chain off every asynchronous round trip
 *                   (chunk 64 or 16, bf16 x and q, m = 64, d in {64, 128}).
 *   SPLIT_REG8      as SPLIT_REG with 8 slots per CTA over a cluster of 8 CTAs:
 *                   half the tensor work on each CTA's chain; needs B*H clusters
 *                   of 8 SMs within one GPC each.
 * An explicit choice that cannot run the shape returns LATTICE_ERR_UNSUPPORTED.
 * All tensor-core choices compute the same chunked form; they differ only in
 * fp32 summation order. */
typedef enum {
    LATTICE_IMPL_AUTO = 0,
    LATTICE_IMPL_SIMT = 1,
    LATTICE_IMPL_TCGEN05 = 2,
    LATTICE_IMPL_TCGEN05_SPLIT = 3,
    LATTICE_IMPL_SPLIT_REG = 4,
    LATTICE_IMPL_SPLIT_REG8 = 5
} lattice_impl;

/* Which kernel LATTICE_IMPL_AUTO runs for a chunked scan of B x H sequences of
 * this shape: SPLIT_REG when it applies (chunk 64 or 16, m = 64) and the current
 * device holds B*H of its 4-CTA clusters at once, else TCGEN05 when it applies,
 * else SIMT (chunk_size 1 is always SIMT). Host function; launches nothing
 * (without a device it assumes the 37 clusters of a 148-SM part). */
lattice_impl lattice_chunk_impl(int B, int H, int m, int d, int chunk_size, lattice_dtype x_dtype,
                                lattice_dtype q_dtype);

/* Whole-sequence forward (the paper's lattice_compress, Appendix D).
 * Reads S0, writes the final state to S_out (S_out == S0 is allowed: the
 * update is then in place; any other overlap between outputs and inputs is
 * LATTICE_ERR_INVALID_ARG) and the read-out of every token to y.
 * chunk_size = 1: exact recurrence; chunk_size > 1: Eq. 17 chunked form.
 * T = 0 copies S0 to S_out and writes nothing else. */
lattice_status lattice_scan_fwd(const void *x, lattice_dtype x_dtype, const float *c,
                                const void *q, lattice_dtype q_dtype, const float *mu,
                                const float *eta, const float *S0, float *S_out, float *y,
                                int B, int T, int H, int m, int d, int chunk_size,
                                lattice_mode mode, void *stream);

/* Chunk form for chunk_size > 1: a linearisation (§3.4.1), optionally OR'ed with
 * LATTICE_CHUNK_NORM_AT_BOUNDARY.
 *   LATTICE_CHUNK_LIN2  Eq. 17 (recurrence_linear2), the default: within a chunk
 *                       each token's gate g = beta (mu + eta hhat khat) scales the
 *                       running slot.
 *   LATTICE_CHUNK_LIN1  eq. recurrence_linear1: the forget part beta mu scales
 *                       the running slot and the projection part beta eta hhat khat
 *                       the chunk-start slot (its chunk form is eq. chunkwise_OSR).
 *   LATTICE_CHUNK_NORM_AT_BOUNDARY  the normalisation ablation of Appendix C
 *                       ("Per-token vs. Per-chunk Normalization"): no per-token
 *                       normaliser inside a chunk (beta = 1); every slot is
 *                       projected onto the unit sphere after each chunk, once the
 *                       chunk's read-outs are done. With chunk_size 1 this is the
 *                       exact recurrence.
 * LIN1 and NORM_AT_BOUNDARY run on the CUDA-core kernel only: tensor-core choices
 * return LATTICE_ERR_UNSUPPORTED, and AUTO takes the CUDA-core kernel. */
typedef enum {
    LATTICE_CHUNK_LIN2 = 0,
    LATTICE_CHUNK_LIN1 = 1,
    LATTICE_CHUNK_NORM_AT_BOUNDARY = 2
} lattice_chunk_form;

/* As lattice_scan_fwd, with an explicit kernel choice (see lattice_impl). */
lattice_status lattice_scan_fwd_impl(const void *x, lattice_dtype x_dtype, const float *c,
                                     const void *q, lattice_dtype q_dtype, const float *mu,
                                     const float *eta, const float *S0, float *S_out, float *y,
                                     int B, int T, int H, int m, int d, int chunk_size,
                                     lattice_mode mode, lattice_impl impl, void *stream);

/* As lattice_scan_fwd_impl, with the chunk form (see lattice_chunk_form; values 0-3;
 * the linearisation is ignored for chunk_size 1). Any other form is
 * LATTICE_ERR_INVALID_ARG. */
lattice_status lattice_scan_fwd_ex(const void *x, lattice_dtype x_dtype, const float *c,
                                   const void *q, lattice_dtype q_dtype, const float *mu,
                                   const float *eta, const float *S0, float *S_out, float *y,
                                   int B, int T, int H, int m, int d, int chunk_size,
                                   lattice_mode mode, lattice_chunk_form form, lattice_impl impl,
                                   void *stream);

/* Backward pass of the similarity-objective scan (exact recurrence for
 * chunk_size 1, Eq. 17 otherwise). The paper prints no backward formulas; this is
 * the reverse-mode derivative of the forward of lattice_scan_fwd with
 * LATTICE_SIM and LATTICE_CHUNK_LIN2, for the scalar loss
 *     L = sum_t dy_t . y_t + dS_T . S_T.
 * Inputs as for lattice_scan_fwd (same layouts and dtypes), plus
 *   dy [B][T][H][d] fp32 (required when T > 0) and dS_T [B][H][m][d] fp32 or NULL (0).
 * Outputs (fp32, device, the inputs' layouts, written in full): dx, dc, dq, dmu,
 *   deta (may be NULL; not written when eta is NULL, i.e. eta = 1) and dS0.
 * States are rebuilt by recomputation from checkpoints every seg_tokens tokens
 * (0 selects the default: the smallest multiple of chunk_size that is >= 64; any
 * other value must be a positive multiple of chunk_size, else
 * LATTICE_ERR_INVALID_ARG). workspace is caller-owned device memory of at least
 * lattice_scan_bwd_workspace_bytes(...) bytes, 16-byte aligned; the call
 * overwrites it and keeps no pointer after it returns (the kernel runs on
 * `stream`). Outputs must not overlap inputs, each other or the workspace
 * (LATTICE_ERR_INVALID_ARG). m <= 128 (larger m: LATTICE_ERR_UNSUPPORTED).
 * Kernels: chunk sizes 2..64 with d in {32, 64, 128}, and x, dy, dx on 16-byte
 * boundaries, run a chunk-parallel kernel: a forward sweep stores every chunk-start
 * state in the workspace, then each chunk, last to first, is differentiated as a whole
 * (matrix products on the tensor cores in tf32 with a hi/lo split of each operand,
 * about fp32 accuracy), and only the state adjoint passes from chunk to chunk;
 * seg_tokens is checked but not used. Other shapes (the exact recurrence included)
 * run token by token on CUDA cores with the segment checkpoints described above.
 * Both are deterministic: sums across CTAs are taken in a fixed order. */
lattice_status lattice_scan_bwd(const void *x, lattice_dtype x_dtype, const float *c,
                                const void *q, lattice_dtype q_dtype, const float *mu,
                                const float *eta, const float *S0, const float *dy,
                                const float *dS_T, float *dx, float *dc, float *dq, float *dmu,
                                float *deta, float *dS0, void *workspace, size_t workspace_bytes,
                                int B, int T, int H, int m, int d, int chunk_size, int seg_tokens,
                                void *stream);

/* Workspace bytes lattice_scan_bwd needs for this shape on the current device: the
 * token kernel's B*H*G*(n_seg - 1 + seg_tokens)*ceil(m/G)*d*4 with
 * n_seg = ceil(T/seg_tokens) (seg_tokens as resolved by lattice_scan_bwd) and G the
 * CTAs per sequence it uses (G = 1 when the batch fills the device's SMs; up to 4
 * otherwise), and, where the chunk-parallel kernel serves the shape, the larger of
 * that and its B*H*ceil(m/16)*ceil(T/chunk)*16*d*4 (every chunk-start state), so that
 * either kernel can run. Returns 0 for arguments lattice_scan_bwd would reject. Host
 * function; launches nothing. */
size_t lattice_scan_bwd_workspace_bytes(int B, int T, int H, int m, int d, int chunk_size,
                                        int seg_tokens);

/* Backward pass that allocates nothing, for callers that cannot call cudaMalloc:
 * for example a plug-in running inside a host application that hands out every
 * byte of device memory through its own pool, or a process that reserved the
 * device's memory up front and may not ask the driver for more. The paper has no
 * counterpart; this is a packaging of lattice_scan_bwd.
 *
 * Arguments, layouts, results and errors are those of lattice_scan_bwd without the
 * workspace: the scratch it needs lives in one static device array of
 * LATTICE_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits. A shape whose workspace
 * (lattice_scan_bwd_workspace_bytes) exceeds that size returns
 * LATTICE_ERR_UNSUPPORTED before any device work. The caller still allocates the
 * inputs and outputs; the call itself makes no allocation.
 *
 * The first call in each CUDA context (the device's primary context, or a context
 * the caller created and made current) looks up the array's device address in that
 * context with cudaGetSymbolAddress and caches it under the context's unique id; make
 * that first call before any stream capture. Every call shares the one array:
 * calls that overlap on the GPU (on different streams, or from different host
 * threads without ordering) race and corrupt each other's results, so order them. Nothing needs clearing between calls: the kernel
 * writes every scratch word before it reads it. */
#define LATTICE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

lattice_status lattice_scan_bwd_noalloc(const void *x, lattice_dtype x_dtype, const float *c,
                                        const void *q, lattice_dtype q_dtype, const float *mu,
                                        const float *eta, const float *S0, const float *dy,
                                        const float *dS_T, float *dx, float *dc, float *dq,
                                        float *dmu, float *deta, float *dS0, int B, int T, int H,
                                        int m, int d, int chunk_size, int seg_tokens, void *stream);

/* One decode step: the exact recurrence for one new token per (b,h), state
 * updated in place (constant work per token, §1-§2 of the paper).
 *   S [B][H][m][d] in/out, x [B][H][d], c [B][H][m], q [B][H][m],
 *   mu [B][H], eta [B][H] or NULL, y [B][H][d] out. */
lattice_status lattice_step(float *S, const void *x, lattice_dtype x_dtype, const float *c,
                            const void *q, lattice_dtype q_dtype, const float *mu,
                            const float *eta, float *y, int B, int H, int m, int d,
                            lattice_mode mode, void *stream);

/* Read-out without an update: y[b][h][:] = sum_i q[b][h][i] S[b][h][i][:]
 * (§2 eq. LA memory read-out; Appendix D y = q @ S). S [B][H][m][d],
 * q [B][H][m], y [B][H][d]. */
lattice_status lattice_readout(const float *S, const void *q, lattice_dtype q_dtype, float *y,
                               int B, int H, int m, int d, void *stream);

/* ---- Gated linear recurrence
 *
 * The linear recurrence that each slot of the chunked form runs (Eq. 17: s <- g s +
 * kappa x), without the projection and the normaliser, for layers that mix both kinds of
 * state: per (batch b, head h, channel j), for t = 1..len_b,
 *     h_t = a_t h_{t-1} + s(a_t) x_t,     y_t = h_t.
 * Gate:  LATTICE_GATE_VALUE  a = z, with |a| <= 1 (larger gates are not supported: the
 *                            products of a run may overflow);
 *        LATTICE_GATE_LOGIT  a = sigmoid(z)^tau, tau > 0. An infinite z is a gate of
 *                            exactly 0 or 1.
 * Write: LATTICE_WRITE_PLAIN s = 1; LATTICE_WRITE_LEAKY s = 1 - a; LATTICE_WRITE_UNIT
 *        s = sqrt(max(0, 1 - a^2)), which keeps the variance of independent unit inputs.
 *
 * Layouts: x [B][T][H][d]; z [B][T][H][d], or [B][T][H] with z_per_head != 0 (then d in
 * {16, 32, 64, 128}); h0, h_out [B][H][d] fp32, row-major; y [B][T][H][d] in x's type. x,
 * z and dy may be slices of wider rows: their batch and token strides are given in
 * elements (>= 0), a token's own H*d (or H) elements are contiguous; the bytes between
 * rows must be readable, whatever they hold. Every output is contiguous. x: fp32, bf16 or
 * fp16; z: fp32 or x's type. Arithmetic and state are fp32 whatever the types; y and the
 * gradients are rounded once.
 * Sizes: B, H, d >= 1, T >= 0; H*d and T up to 2^30.
 * lengths (int32 [B], device, or NULL for T each) gives every sequence its own length,
 * taken into 0..T. Tokens behind it are not read: their y and gradients are written as
 * zero, and h_out is the state at the sequence's own end (h0 for a length of 0).
 * Results do not depend on the run: every sum has a fixed order. */
typedef enum { LATTICE_GATE_VALUE = 0, LATTICE_GATE_LOGIT = 1 } lattice_gate;
typedef enum { LATTICE_WRITE_PLAIN = 0, LATTICE_WRITE_LEAKY = 1, LATTICE_WRITE_UNIT = 2 } lattice_write;

/* Whole sequences. h0 may be NULL (0). h_out may be NULL or h0 (in place); y may be NULL
 * when marks is given. marks (or NULL): device memory of lattice_gated_scan_marks_bytes,
 * 16-byte aligned, filled with the state before every 16th token, for the backward pass.
 * Outputs must not overlap inputs or each other (LATTICE_ERR_INVALID_ARG). Running a
 * sequence in pieces, each from the state of the one before, gives the same recurrence. */
lattice_status lattice_gated_scan_fwd(const void *x, lattice_dtype x_dtype,
                                      long long x_batch_stride, long long x_token_stride,
                                      const void *z, lattice_dtype z_dtype,
                                      long long z_batch_stride, long long z_token_stride,
                                      int z_per_head, const float *h0, float *h_out, void *y,
                                      float *marks, const int *lengths, int B, int T, int H, int d,
                                      lattice_gate gate, lattice_write write, float tau,
                                      void *stream);

/* Bytes of marks for this shape (0 for T = 0 or sizes the scan rejects). Host function. */
size_t lattice_gated_scan_marks_bytes(int B, int T, int H, int d);

/* Backward pass for L = sum_t dy_t . y_t + dh_T . h_len. x, z, lengths and the forms as in
 * the forward call that filled marks (marks carries h0, which is therefore not an argument);
 * dy in x's type, dh_T [B][H][d] fp32 or NULL (0). Writes dx (x's type), dz (z's type and
 * shape; a gate per head collects its d channels) and dh0 [B][H][d] fp32, all contiguous and
 * in full. Where s = 0 (|a| >= 1) the unit write passes no gradient to its gate. */
lattice_status lattice_gated_scan_bwd(const void *x, lattice_dtype x_dtype,
                                      long long x_batch_stride, long long x_token_stride,
                                      const void *z, lattice_dtype z_dtype,
                                      long long z_batch_stride, long long z_token_stride,
                                      int z_per_head, const void *dy, long long dy_batch_stride,
                                      long long dy_token_stride, const float *marks,
                                      const float *dh_T, void *dx, void *dz, float *dh0,
                                      const int *lengths, int B, int T, int H, int d,
                                      lattice_gate gate, lattice_write write, float tau,
                                      void *stream);

/* One token: h_out = a h + s(a) x, y = h_out in x's type. h, h_out [B][H][d] fp32 (h_out ==
 * h: in place); x [B][H][d], z [B][H][d] or [B][H], with batch strides as above. */
lattice_status lattice_gated_step(const float *h, float *h_out, const void *x,
                                  lattice_dtype x_dtype, long long x_batch_stride, const void *z,
                                  lattice_dtype z_dtype, long long z_batch_stride, int z_per_head,
                                  void *y, int B, int H, int d, lattice_gate gate,
                                  lattice_write write, float tau, void *stream);

/* ---- Norms after and before a block
 *
 * What surrounds a recurrence in a layer: the norm of its read-out with the gate on it (the
 * paper's block has a GeLU gate after the read-out, Appendix C), and after the output
 * projection the scaled residual and the next block's norm. Per row of D elements:
 *     u = y / sqrt(mean y^2 + eps)       (u = y with post_norm 0)
 *     v = scale u w_post act(gate)       (w_post, gate: 1 where NULL)
 *     r = residual + v                   (r = v without a residual)
 *     n = r / sqrt(mean r^2 + eps) w_pre (if wanted)
 * Types: `dtype` is that of gate and n; y, residual and r, and the weights (both) are of it
 * or fp32. r has the residual's type, or dtype without one. Arithmetic is fp32 and n is
 * formed from r before its rounding; the sum of a row's squares must be within fp32's range.
 * Rows: N rows of D contiguous elements, 1 <= D <= 16384, 0 <= N < 2^31. Inputs come in
 * groups of G rows (N a multiple of G), contiguous within a group, with the given stride
 * in elements (0 to 2^31 - 1) between groups: G = 1 for rows of any stride, G = H for heads
 * [B*T][H][D] cut out of wider tokens; what is between groups must be readable, whatever it
 * holds. Outputs are contiguous.
 * act: applied to the gate; NONE: the gate is not allowed. eps > 0. */
typedef enum { LATTICE_ACT_NONE = 0, LATTICE_ACT_SIGMOID = 1, LATTICE_ACT_SILU = 2, LATTICE_ACT_GELU = 3 } lattice_act;

/* r_out may be the residual (same buffer, contiguous): the residual stream is then updated
 * in place. n_out NULL: n is not formed (w_pre must then be NULL). */
lattice_status lattice_block_norm_fwd(const void *y, lattice_dtype y_dtype, long long y_stride,
                                      const void *gate, long long gate_stride, const void *residual,
                                      lattice_dtype residual_dtype, long long residual_stride,
                                      const void *w_post, const void *w_pre, lattice_dtype w_dtype,
                                      void *r_out, void *n_out, lattice_dtype dtype, long long N,
                                      int G, int D, lattice_act act, int post_norm, float scale,
                                      float eps, void *stream);

/* Bytes of workspace of lattice_block_norm_bwd on the current device (0 for sizes it
 * rejects). Host function. */
size_t lattice_block_norm_bwd_workspace_bytes(long long N, int D);

/* Backward pass, recomputing from the forward call's inputs. dr: cotangent of r, in
 * dr_dtype (fp32 or dtype; with a residual, the residual's type), or NULL (0); dn: cotangent
 * of n in dtype, or NULL (n was not formed); at least one is given. Writes dy (y's type),
 * dgate (dtype; required with a gate), dresidual (the residual's type; required with a
 * residual), all contiguous, and the weights' gradients dw_post, dw_pre [D] fp32, each NULL
 * where it is not wanted. workspace: lattice_block_norm_bwd_workspace_bytes, 16-byte
 * aligned, needed if a weight's gradient is wanted. Sums over rows are taken in a fixed
 * order for given sizes and device. */
lattice_status lattice_block_norm_bwd(const void *y, lattice_dtype y_dtype, long long y_stride,
                                      const void *gate, long long gate_stride, const void *residual,
                                      lattice_dtype residual_dtype, long long residual_stride,
                                      const void *w_post, const void *w_pre, lattice_dtype w_dtype,
                                      const void *dr, lattice_dtype dr_dtype, long long dr_stride,
                                      const void *dn, long long dn_stride, void *dy, void *dgate,
                                      void *dresidual, float *dw_post, float *dw_pre,
                                      void *workspace, size_t workspace_bytes, lattice_dtype dtype,
                                      long long N, int G, int D, lattice_act act, int post_norm,
                                      float scale, float eps, void *stream);

/* ---- Short causal convolution
 *
 * The convolution of few taps that stands before a recurrence (the paper's block has one on keys and
 * queries, Appendix C), every channel by itself, over the tokens of a sequence:
 *     v_t = bias + sum_k w[k] x_{t-K+1+k},  y_t = act(v_t),  k = 0..K-1.
 * The K-1 inputs before the first token are the state's rows, oldest first, or 0 without one.
 *
 * Layouts: x [B][T][C], w [C][K], bias [C] (or NULL: 0), state [B][K-1][C], row-major; y in x's type
 * and layout. x and dy may be slices of wider rows: batch and token strides in elements (>= 0), a
 * token's C elements contiguous. Outputs are contiguous. x: fp32, bf16 or fp16; w and bias, one type
 * for both, fp32 or x's; the state has x's type. Arithmetic is fp32, results are rounded once.
 * Sizes: B, C >= 1, T >= 0, 1 <= K <= 8; C and T up to 2^30. act: NONE or SILU.
 * lengths (int32 [B], device, or NULL for T each), taken into 0..T: tokens behind a sequence's
 * length are not read, their y and gradients are written as zero, and the state left is that at the
 * sequence's own end. Sums have a fixed order for given sizes and device. */

/* Whole sequences. state_out (or NULL): the last K-1 inputs before each sequence's end, for the next
 * call; it may be the state itself. Other outputs must not overlap inputs or each other. */
lattice_status lattice_short_conv_fwd(const void *x, lattice_dtype x_dtype, long long x_batch_stride,
                                      long long x_token_stride, const void *w, const void *bias,
                                      lattice_dtype w_dtype, const void *state, void *state_out, void *y,
                                      const int *lengths, int B, int T, int C, int K, lattice_act act,
                                      void *stream);

/* Bytes of workspace of lattice_short_conv_bwd on the current device (0 for sizes it rejects). Host
 * function. */
size_t lattice_short_conv_bwd_workspace_bytes(int B, int T, int C, int K);

/* Backward pass for L = sum dy . y + sum dstate_out . state_out, from the forward call's inputs; dy
 * in x's type, dstate_out [B][K-1][C] in x's type or NULL (0). Writes dx and dstate (x's type; dstate
 * only with a state, or NULL), dw [C][K] and dbias [C] (fp32, each NULL where it is not wanted).
 * workspace: lattice_short_conv_bwd_workspace_bytes, 16-byte aligned, needed for dw or dbias. */
lattice_status lattice_short_conv_bwd(const void *x, lattice_dtype x_dtype, long long x_batch_stride,
                                      long long x_token_stride, const void *w, const void *bias,
                                      lattice_dtype w_dtype, const void *state, const void *dy,
                                      long long dy_batch_stride, long long dy_token_stride,
                                      const void *dstate_out, void *dx, float *dw, float *dbias,
                                      void *dstate, void *workspace, size_t workspace_bytes,
                                      const int *lengths, int B, int T, int C, int K, lattice_act act,
                                      void *stream);

/* One token: y from the state and x [B][C]; state_out is the state without its oldest row and with x
 * as its last (state_out == state: in place). */
lattice_status lattice_short_conv_step(const void *state, void *state_out, const void *x,
                                       lattice_dtype x_dtype, long long x_batch_stride, const void *w,
                                       const void *bias, lattice_dtype w_dtype, void *y, int B, int C,
                                       int K, lattice_act act, void *stream);

/* ---- Selective state space scan
 *
 * The gated linear recurrence with N states per channel, whose decay, write and read are chosen by
 * the token. Per (batch, channel e, state n), for t = 1..len_b, with
 * dt_t = softplus(dt_raw + dt_bias[e]) (or dt_raw + dt_bias[e] with softplus 0):
 *     h_t[n] = exp(dt_t A[e][n]) h_{t-1}[n] + dt_t x_t b_t[n]
 *     y_t = (sum_n c_t[n] h_t[n] + skip[e] x_t) silu(z_t)          (no last factor without z)
 * b and c belong to a group of E/G neighbouring channels. dt_t A <= 0 is expected: growing states
 * may overflow, also where the whole sequence's would not.
 *
 * Layouts: x, z, dt [B][T][E]; b, c [B][T][G][N]; A [E][N], skip, dt_bias [E], h0, h_out [B][E][N]
 * fp32, row-major. x, z, dt, b, c and dy may be slices of wider rows: batch and token strides in
 * elements (>= 0), a token's own E (or G*N) elements contiguous. x, z, b, c, y and dy have one type
 * (fp32, bf16 or fp16), dt it or fp32. Arithmetic and states are fp32 whatever the types; y and the
 * gradients are rounded once. Outputs are contiguous.
 * Sizes: B, E, N, G >= 1, E a multiple of G, N <= 128, T >= 0; E and T up to 2^30.
 * lengths: as for the gated recurrence: tokens behind a sequence's length are not read, their y and
 * gradients are zero, and h_out is the state at the sequence's own end.
 * workspace: lattice_selective_scan_workspace_bytes on the current device (which may be 0), 16-byte
 * aligned. Results do not depend on the run: every sum has a fixed order for given sizes and device.
 * Memory: marks take N/2 bytes per element of x, the backward pass's workspace some N P/128 more for
 * its sums of db and dc (P: N padded to a power of two, 8 at least; up to 4 times as much with few
 * channels per group). 8 x 4096 tokens of 2048 channels: 0.5 and 0.13 GiB with 16 states, 4 and 8
 * GiB with 128.
 * Inputs that are not finite: where the formula has an infinity, states and what is read from them
 * may be NaN instead. */

/* Whole sequences. h0 NULL: 0; h_out NULL or h0 (in place); z, skip, dt_bias, lengths may be NULL; y
 * may be NULL when marks is given. marks (or NULL): device memory of
 * lattice_selective_scan_marks_bytes, 16-byte aligned, for the backward pass: filled with the state
 * before every 8th token up to each sequence's end. */
lattice_status lattice_selective_scan_fwd(const void *x, lattice_dtype x_dtype, long long x_batch_stride,
                                          long long x_token_stride, const void *dt, lattice_dtype dt_dtype,
                                          long long dt_batch_stride, long long dt_token_stride,
                                          const float *A, const void *b, long long b_batch_stride,
                                          long long b_token_stride, const void *c, long long c_batch_stride,
                                          long long c_token_stride, const float *skip, const void *z,
                                          long long z_batch_stride, long long z_token_stride,
                                          const float *dt_bias, int softplus, const float *h0, float *h_out,
                                          void *y, float *marks, const int *lengths, void *workspace,
                                          size_t workspace_bytes, int B, int T, int E, int N, int G,
                                          void *stream);

/* Bytes of marks, and of workspace for one direction, for these sizes (0 also for sizes the scan
 * rejects). Host functions. */
size_t lattice_selective_scan_marks_bytes(int B, int T, int E, int N);
size_t lattice_selective_scan_workspace_bytes(int B, int T, int E, int N, int G, int backward);

/* Backward pass for L = sum_t dy_t . y_t + dh_T . h_len. The inputs are those of the forward call
 * that filled marks (which carries h0); dh_T [B][E][N] fp32 or NULL (0). Writes dx, dz (z only), db,
 * dc (x's type), ddt (dt's type: the gradient of dt_raw), dA [E][N], dskip, ddt_bias [E] (each of
 * these two NULL where it is not wanted) and dh0 [B][E][N] (fp32), all contiguous and in full. */
lattice_status lattice_selective_scan_bwd(const void *x, lattice_dtype x_dtype, long long x_batch_stride,
                                          long long x_token_stride, const void *dt, lattice_dtype dt_dtype,
                                          long long dt_batch_stride, long long dt_token_stride,
                                          const float *A, const void *b, long long b_batch_stride,
                                          long long b_token_stride, const void *c, long long c_batch_stride,
                                          long long c_token_stride, const float *skip, const void *z,
                                          long long z_batch_stride, long long z_token_stride,
                                          const float *dt_bias, int softplus, const void *dy,
                                          long long dy_batch_stride, long long dy_token_stride,
                                          const float *marks, const float *dh_T, void *dx, void *ddt,
                                          float *dA, void *db, void *dc, float *dskip, void *dz,
                                          float *ddt_bias, float *dh0, const int *lengths, void *workspace,
                                          size_t workspace_bytes, int B, int T, int E, int N, int G,
                                          void *stream);

/* One token: h_out from h (h_out == h: in place) and y [B][E]; x, z, dt [B][E], b, c [B][G][N], with
 * batch strides as above. */
lattice_status lattice_selective_step(const float *h, float *h_out, const void *x, lattice_dtype x_dtype,
                                      long long x_batch_stride, const void *dt, lattice_dtype dt_dtype,
                                      long long dt_batch_stride, const float *A, const void *b,
                                      long long b_batch_stride, const void *c, long long c_batch_stride,
                                      const float *skip, const void *z, long long z_batch_stride,
                                      const float *dt_bias, int softplus, void *y, int B, int E, int N,
                                      int G, void *stream);

/* ---- Layer norm
 *
 * The norm before a block whose rows are also centred, with the residual that they are added to:
 *     r = residual + x              (rounded to the residual's type; r = x without a residual)
 *     n = (r - mean r) / sqrt(mean (r - mean r)^2 + eps) w + b
 * n is formed from r as it is kept. w, b [D] or NULL (1, 0), one type for both. Types, rows, strides,
 * sizes and eps are those of the block norms: `dtype` is n's; x, the residual and r (the residual's
 * type) and the weights are of it or fp32. */

/* r_out is given exactly with a residual, which it may be (same buffer, contiguous). */
lattice_status lattice_layer_norm_fwd(const void *x, lattice_dtype x_dtype, long long x_stride,
                                      const void *residual, lattice_dtype residual_dtype,
                                      long long residual_stride, const void *w, const void *b,
                                      lattice_dtype w_dtype, void *r_out, void *n_out, lattice_dtype dtype,
                                      long long N, int G, int D, float eps, void *stream);

/* Bytes of workspace of lattice_layer_norm_bwd on the current device (0 for sizes it rejects). Host
 * function. */
size_t lattice_layer_norm_bwd_workspace_bytes(long long N, int D);

/* Backward pass from the normed rows r (the forward call's r_out, or x without a residual): dn is n's
 * cotangent, dr that of r from elsewhere (r's type, or NULL: 0). Writes dr_out, the gradient of r and
 * so of the residual and of x, in r's type; dx (or NULL), the same in x's type; and dw, db [D] fp32
 * (each NULL where it is not wanted; dw only with w). workspace: lattice_layer_norm_bwd_workspace_bytes,
 * 16-byte aligned, needed for dw or db. Sums over rows have a fixed order for given sizes and device. */
lattice_status lattice_layer_norm_bwd(const void *r, lattice_dtype r_dtype, long long r_stride,
                                      const void *dn, long long dn_stride, const void *dr,
                                      long long dr_stride, const void *w, lattice_dtype w_dtype,
                                      void *dr_out, void *dx, lattice_dtype x_dtype, float *dw, float *db,
                                      void *workspace, size_t workspace_bytes, lattice_dtype dtype,
                                      long long N, int G, int D, float eps, void *stream);

/* Synchronises `stream`, returns LATTICE_ERR_TIMEOUT if any kernel since the
 * last call gave up a bounded wait (and clears the flag), LATTICE_ERR_CUDA if
 * the stream reports an error, else LATTICE_OK. */
lattice_status lattice_get_device_status(void *stream);

/* Failure-detection self-test (the paper has no counterpart): launches one warp
 * that waits, with the same bounded device-side wait the tensor-core kernels use,
 * on an mbarrier that nothing ever completes. After limit_ns nanoseconds (1 ns to
 * 1 s; else LATTICE_ERR_INVALID_ARG, nothing launched) the wait gives up, sets the
 * device status word and the kernel returns, so the next
 * lattice_get_device_status(stream) returns LATTICE_ERR_TIMEOUT (and clears the
 * word) while the CUDA context stays usable. Asynchronous on `stream`. */
lattice_status lattice_selftest_bounded_wait(unsigned long long limit_ns, void *stream);

/* Name and description of the last CUDA error the library saw on this host
 * thread when a call returned LATTICE_ERR_CUDA ("" if none). The text is
 * owned by the library and stays valid until the next call on this thread. */
const char *lattice_last_cuda_error(void);

/* Static English text for a status code. */
const char *lattice_status_string(lattice_status s);

/* Library version, major*10000 + minor*100 + patch. */
int lattice_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LATTICE_H_ */

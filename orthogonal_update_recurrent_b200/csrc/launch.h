// launch.h -- host interface between the C ABI (lattice_abi.cu) and the kernel
// families. Each family is compiled in a translation unit of its own (tu_*.cu), so
// that the units build in parallel and each is optimised as a whole; this header
// carries no device code.
#pragma once
#include <cuda_runtime.h>

#include "../../include/lattice.h"
#include "args.h"

namespace lattice {

// lattice_abi.cu: error recording and device queries shared by every unit
lattice_status cuda_fail(cudaError_t e);
lattice_status launch_status();
int sm_count();
// Lets a kernel be launched with up to `most` bytes of dynamic shared memory. The limit belongs to
// the kernel on its device, whoever calls: it is set to the most that any of the kernel's launches
// takes, so that a launch never meets the smaller limit of another host thread's call.
template <class... A>
cudaError_t allow_shared(void (*kernel)(A...), size_t most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}
// CTAs per sequence for the CUDA-core kernels (a cluster when > 1)
int cluster_split(int B, int H, int m);

// tu_simt_exact.cu, tu_simt_chunked.cu: CUDA-core scans, exact or chunked (either linearisation)
lattice_status launch_scan_simt_exact(const ScanArgs& a, int d, bool dec, cudaStream_t st);
lattice_status launch_scan_simt_chunked(const ScanArgs& a, int d, bool dec, bool lin1, cudaStream_t st);
inline lattice_status launch_scan_simt(const ScanArgs& a, int d, bool chunked, bool dec, bool lin1, cudaStream_t st) {
    return chunked ? launch_scan_simt_chunked(a, d, dec, lin1, st) : launch_scan_simt_exact(a, d, dec, st);
}

// tu_step.cu: decode step and read-out
lattice_status launch_step(const StepArgs& a, int d, bool dec, cudaStream_t st);
lattice_status launch_readout(const ReadoutArgs& a, int d, cudaStream_t st);

// tu_bwd.cu: backward pass (a.G, a.spc set by the caller)
lattice_status launch_bwd(const BwdArgs& a, int d, cudaStream_t st);
lattice_status launch_chunk_bwd(const BwdArgs& a, int d, cudaStream_t st);

// tu_tc.cu: tensor-core chunked scans
bool tc_supported(lattice_impl impl, int m, int d, int chunk, bool x_bf16, bool q_bf16);
lattice_status launch_tc(lattice_impl impl, const ScanArgs& a, int d, cudaStream_t st);
// clusters of 4 CTAs of the register-chain kernel the current device holds at once
int reg_cluster_capacity(int d);

// tu_gated_fwd_*.cu, tu_gated_bwd_*.cu: gated linear recurrence, a unit per type of x
// (ctiles, K set by the launch). form = 3 * gate form + write form (gated.cuh); vec: every
// row can be read in aligned vectors of the elements that a lane has
constexpr int kGatedFwdVec = 2, kGatedBwdVec = 2, kGatedHeadVec = 4, kStepVec = 4;
namespace gated {
template <class XT> lattice_status launch_fwd(GatedArgs a, int form, bool vec, cudaStream_t st);
template <class XT> lattice_status launch_step(const GatedArgs& a, int form, bool vec, cudaStream_t st);
template <class XT> lattice_status launch_bwd(GatedArgs a, int form, bool vec, cudaStream_t st);
}  // namespace gated

// tu_norm_*.cu: norms after and before a block, a unit per type of the call (tpr, K set by the
// launch). mode: rows and weights can be read in aligned vectors of 8 elements (kNormVec), rows in
// vectors that start where a vector does (kNormShift), or one by one (kNormOdd); groups
// (or null): how many rows of weight gradients the backward pass leaves in the workspace
namespace norm {
template <class XT> lattice_status launch_norm(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);
// tu_lnorm_*.cu: layer norm (y: x or backward r; w_post, w_pre: its weight and bias)
template <class XT> lattice_status launch_layer(bool bwd, NormArgs a, int mode, int* groups, cudaStream_t st);
}  // namespace norm
int norm_parts(long long N, int D);  // at most so many
int layer_parts(long long N, int D);
lattice_status launch_norm_dw(const NormArgs& a, int groups, float* dw_post, float* dw_pre, cudaStream_t st);

// conv_*.cu: short convolution, a unit per type of x (no waits in it, and so no status word). V: channels
// per thread, 4, 2 or 1, as many as rows can be read in vectors of
namespace conv {
template <class XT> lattice_status launch(const ConvArgs& a, int what, int V, cudaStream_t st);
}  // namespace conv

// sel_fwd_*.cu, sel_bwd_*.cu: selective scan, a unit per type of x (no waits either). S: states per
// lane; W: warps of a CTA, 8 or 2
namespace selective {
template <class XT> lattice_status launch_fwd(const SelArgs& a, int S, int W, cudaStream_t st);
template <class XT> lattice_status launch_step(const SelArgs& a, cudaStream_t st);
template <class XT> lattice_status launch_bwd(const SelArgs& a, int W, cudaStream_t st);
}  // namespace selective

// each unit's device status word (read, and zeroed when set)
cudaError_t status_simt_exact(unsigned int* v);
cudaError_t status_simt_chunked(unsigned int* v);
cudaError_t status_step(unsigned int* v);
cudaError_t status_bwd(unsigned int* v);
cudaError_t status_tc(unsigned int* v);
cudaError_t status_norm_f32(unsigned int* v);
cudaError_t status_norm_bf16(unsigned int* v);
cudaError_t status_norm_f16(unsigned int* v);
cudaError_t status_lnorm_f32(unsigned int* v);
cudaError_t status_lnorm_bf16(unsigned int* v);
cudaError_t status_lnorm_f16(unsigned int* v);
cudaError_t status_gated_fwd_f32(unsigned int* v);
cudaError_t status_gated_fwd_bf16(unsigned int* v);
cudaError_t status_gated_fwd_f16(unsigned int* v);
cudaError_t status_gated_bwd_f32(unsigned int* v);
cudaError_t status_gated_bwd_bf16(unsigned int* v);
cudaError_t status_gated_bwd_f16(unsigned int* v);

}  // namespace lattice

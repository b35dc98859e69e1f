// kernels.h -- launch interface between the C-ABI host code and the gfx950 kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sss {

// Compute units of `device` / of the current device, cached (api.cpp); -1 if it cannot be queried.
int device_cus(int device);
int current_device_cus();

// Launch plan of the selective scan (chosen on the host, see selective_scan.hip).
struct SelPlan {
  int segments;      // time segments S (S > 1: segment states, carry, then outputs)
  int64_t seg_len;   // steps per segment (multiple of the load batch)
  size_t ws_state, ws_dsum, ws_bc, ws_total;  // workspace offsets / total bytes
};

struct SelArgs {
  const void* x;
  const void* delta;
  const float* A;
  const float* B;
  const float* C;
  const float* Dsk;
  const void* z;
  const float* h0;
  float* y;
  float* h_last;
  int64_t batch, seqlen, dim;
  int dstate;
  int bf16;
  void* workspace;
  const float* delta_bias;  // nullable: added to delta before use
  int softplus;             // step size = softplus(delta (+ bias))
  int exact_zoh;            // input term expm1(delta*A)/A * B instead of delta * B
  int bdl;                  // x/delta/z/y (batch, dim, seqlen), B/C (batch, dstate, seqlen)
  float* states;            // nullable: the segment entering states [S][batch][dstate][dim] live
                            // here instead of in the workspace (kept for the backward pass)
};

// max_ws > 0: at most max_ws bytes of workspace (fewer segments if the usual plan needs more)
SelPlan plan_selective(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int num_cus, bool bdl = false,
                       size_t max_ws = 0);
hipError_t launch_selective(const SelArgs& a, const SelPlan& plan, hipStream_t stream);
// single-pass form with the workgroup-level pair scan (chunk_scan.hip): which calls it takes,
// and the launch (no workspace)
bool chunk_scan_supported(const SelArgs& a);
hipError_t launch_chunk_scan(const SelArgs& a, hipStream_t stream);
// the whole forward call (api.cpp): validation, plan (workspace at most max_ws bytes when
// max_ws > 0), launch; returns an sss_status
int sel_fwd_impl(const void* x, const void* delta, const float* A, const float* B, const float* C,
                 const float* D_skip, const void* z, const float* h0, float* y, float* h_last,
                 const float* delta_bias, unsigned flags, int64_t batch, int64_t seqlen, int64_t dim,
                 int64_t dstate, int io_dtype, void* workspace, size_t workspace_bytes, size_t max_ws,
                 void* stream, bool save_states = false, float* states = nullptr, size_t states_bytes = 0);
// how the forward kernels walk the rows: 0 time-major; channel-major 1 one step per access,
// 2 16-byte pieces per lane, 3 tiles staged through LDS
int selective_row_mode(const SelArgs& a, const SelPlan& plan);
// pass 1 + carry only: the workspace's state slots hold the state entering each segment
hipError_t launch_segment_states(const SelArgs& a, const SelPlan& plan, hipStream_t stream);
// the state before every 2^kshift-th step of every segment, into
// ckpt[s][batch][channel group][j][dstate + 1][64 lanes] (ceil(dim / 64) groups); with adj_mu
// (more than one segment) also the adjoint of every segment folded from zero at its end into
// adj_mu[s][batch][dstate][dim], dy (batch, seqlen, dim) being the output gradient, and every
// segment's delta sum into the workspace's sums.  Without `local`, after
// launch_segment_states (or with states kept by the forward call): the checkpoints are the
// states.  With `local` (adj_mu, more than one segment) every segment starts from zero: the
// checkpoints hold the states from zero and, in row dstate, the delta sum of the segment's
// steps before them, and the state slots end up holding the entering states (end states
// from zero, then the carry)
hipError_t launch_checkpoints(const SelArgs& a, const SelPlan& plan, float* ckpt, int kshift, int nsub,
                              const float* dy, float* adj_mu, bool local, hipStream_t stream);

// Backward pass of the selective scan (selective_bwd.hip).
struct BwdPlan {
  SelPlan fwd;     // segments of the forward pass (its workspace comes first)
  int K, KC, nsub; // steps per sub-chunk, checkpoint spacing (a multiple of K), checkpoints
                   // per segment
  size_t off_mu, off_ckpt, off_bc, off_pa, off_pd, off_pdb, ws_total;
};

struct BwdArgs {
  SelArgs fwd;  // forward inputs (y / h_last unused)
  const float* dy;
  const float* dh_last;
  float* dx;
  float* ddelta;
  float* dA;
  float* dB;
  float* dC;
  float* dD;
  float* dz;
  float* dh0;
  float* ddelta_bias;  // with the delta front end (fwd.delta_bias / fwd.softplus): d/d bias
  bool states_ready;  // fwd.states already holds the segment entering states (saved by the forward)
};

BwdPlan plan_selective_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int num_cus);
hipError_t launch_selective_bwd(const BwdArgs& a, const BwdPlan& plan, hipStream_t stream);

struct EwPlan {
  int segments;
  int64_t seg_len;
  size_t ws_total;
  int cpl;  // adjacent channels per lane (1, 2 or 4)
};

struct EwArgs {
  const float* x;
  const float* A;
  const float* B;
  const float* C;
  const float* h0;
  float* y;
  float* h_last;
  int64_t batch, seqlen, dim;
  void* workspace;
};

EwPlan plan_elementwise(int64_t batch, int64_t seqlen, int64_t dim, int num_cus);
hipError_t launch_elementwise(const EwArgs& a, const EwPlan& plan, hipStream_t stream);

struct UpdArgs {
  const void* x;
  const void* delta;
  const float* A;
  const float* B;
  const float* C;
  const float* Dsk;
  const void* z;
  float* state;
  float* y;
  int64_t batch, dim;
  int dstate;
  int bf16;
};

hipError_t launch_update(const UpdArgs& a, hipStream_t stream);

struct ConvPlan {
  int segments;
  int64_t seg_len;
  int cpl;  // channels per lane (adjacent), 1 or 8 bytes' worth
};

struct ConvArgs {
  const void* x;
  const float* w;
  const float* bias;
  void* out;
  int64_t batch, seqlen, dim;
  int width;
  int bf16;
  int silu;
};

ConvPlan plan_conv1d(int64_t batch, int64_t seqlen, int64_t dim, bool bf16, int num_cus);
hipError_t launch_conv1d(const ConvArgs& a, const ConvPlan& plan, hipStream_t stream);

// Causal convolution over packed prompts, or one token per row (step), with the inputs before
// them in cache slots (packed_conv.hip).
struct PackedConvArgs {
  const void* x;
  int64_t x_stride;  // elements between tokens
  const float* w;
  const float* bias;
  void* state;           // (slots, width-1, dim), nullable for prompts
  const int32_t* cu;     // nseq + 1 boundaries (prompts)
  const int32_t* sidx;   // nullable: slot of each sequence or row
  const uint8_t* init;   // nullable (prompts): sequences that continue their slot
  void* out;
  int64_t tokens, nseq, slots, dim;
  int width, bf16, silu, step;
};

hipError_t launch_packed_conv(const PackedConvArgs& a, hipStream_t stream);

// Gradients of the causal convolution (conv_bwd.hip).
struct ConvBwdPlan {
  int segments;
  int64_t seg_len;
  int cpl;  // channels per lane
  size_t ws_total;
};

struct ConvBwdArgs {
  const void* x;
  int64_t x_row, x_batch;  // strides in elements
  const float* w;
  const float* bias;
  const void* dout;
  void* dx;
  int64_t dx_row, dx_batch;
  float* dw;
  float* db;
  void* workspace;
  int64_t batch, seqlen, dim;
  int width, bf16, dout_bf16, dx_bf16, silu;
};

ConvBwdPlan plan_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, bool bf16, int num_cus);
hipError_t launch_conv_bwd(const ConvBwdArgs& a, const ConvBwdPlan& plan, hipStream_t stream);

// Selective scan over packed prompts (packed_scan.hip) and the decode step on cache slots
// (slot_update.hip; tokens = rows, no boundaries).
struct PackedScanPlan {
  int64_t K;   // tokens per chunk
  int chunks;
  size_t off_end, off_init, off_enter, off_sum, off_flag, ws_total;
};

struct PackedScanArgs {
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dsk;
  const void* z;
  const float* delta_bias;
  float* state;
  const int32_t* cu;
  const int32_t* sidx;
  const uint8_t* init;
  void* y;
  int64_t sx, sd, sz, sb, sc;  // elements between tokens
  int64_t tokens, nseq, slots, dim;
  int dstate, bf16, bc_bf16, y_bf16, softplus;
  void* workspace;
};

PackedScanPlan plan_packed_scan(int64_t tokens, int64_t dim, int64_t dstate, int num_cus);
hipError_t launch_packed_scan(const PackedScanArgs& a, const PackedScanPlan& plan, hipStream_t stream);
hipError_t launch_pscan_carry(const float* A, const float* ends, const float* sums, const int32_t* flags, float* enter,
                              int dstate, int dim, int chunks, hipStream_t stream);
double slot_update_threads(int64_t rows, int64_t dim, int64_t dstate);  // of its launch
hipError_t launch_slot_update(const PackedScanArgs& a, hipStream_t stream);

// Norms around the block (norms.hip).  Pointers marked nullable may be null.
constexpr int64_t kMaxNormDim = 32768;  // elements of a normed row: 1024 lanes of 32
struct NormPlan {
  int nblk;  // workgroups per group of the gradients kernel: rows of partial parameter gradients
  size_t ws_total;
};

struct GatedNormArgs {
  const void* x;
  const void* z;  // nullable: no gate
  const float* w;
  void* out;
  float* rstd;  // (rows, groups): nullable output of the forward, input of the backward
  const void* dout;
  void* dx;
  void* dz;
  float* dw;
  void* workspace;
  int64_t rows, group, groups;
  int64_t sx, sz, sdz;  // elements between rows
  float eps;
  int x_bf16, z_bf16, norm_first;  // out and dout have z's type
};

struct ResNormArgs {
  const void* x;         // backward: nullable without post norm and scale
  const void* residual;  // nullable: zero
  const float* wp;       // nullable: no post norm
  const float* scale;    // nullable: one
  const float* w;
  void* out;
  void* residual_out;  // backward: input
  float* rstd_post;    // nullable in the forward
  float* rstd;
  const void* dout;
  const void* dres_out;  // nullable: zero
  void* dx;
  void* dres;  // nullable
  float* dw;
  float* dwp;
  float* dscale;
  void* workspace;
  int64_t rows, dim;
  int64_t sx, sr;
  float eps, alpha;
  int x_bf16, h_bf16;
};

// fp32: one of the call's tensors is (its kernels take other shapes)
int norm_lanes(int64_t group, bool fp32);  // lanes that share a row of a group
NormPlan plan_norm_bwd(int64_t rows, int64_t group, int64_t groups, int vectors, bool fp32, int num_cus);
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t stream);
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, const NormPlan& plan, hipStream_t stream);
hipError_t launch_res_norm_fwd(const ResNormArgs& a, hipStream_t stream);
hipError_t launch_res_norm_bwd(const ResNormArgs& a, const NormPlan& plan, hipStream_t stream);

// Layer norm (layer_norm.hip).
struct LayerNormArgs {
  const void* x;         // backward: what was normed (the forward's x or residual_out), of the stream's type
  const void* residual;  // nullable: zero
  const float* w;        // nullable: one
  const float* b;        // nullable: zero
  void* out;
  void* residual_out;  // nullable
  float* mean;         // (rows, groups): nullable outputs of the forward, inputs of the backward
  float* rstd;
  const void* dout;
  const void* dres_out;  // nullable: zero
  void* dx;
  void* dres;  // nullable
  float* dw;   // nullable
  float* db;   // nullable
  void* workspace;
  int64_t rows, group, groups;
  int64_t sx, sr;  // elements between rows
  float eps;
  int x_bf16, h_bf16;  // x, out, dout and dx; the residual stream and its gradients
};

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, hipStream_t stream);
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, const NormPlan& plan, hipStream_t stream);

int env_int(const char* name, int dflt);

}  // namespace sss

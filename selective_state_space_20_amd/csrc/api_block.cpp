// api_block.cpp -- the C ABI of the operators around the scan (declared in include/sss.h): the
// packed convolution, scan and their token steps, the convolution's gradients, and the norms
// around the block.
#include "sss.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "api_util.h"
#include "kernels.h"

using namespace sss;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // token numbers are 32-bit on the device
constexpr int64_t kMaxRowDim = (int64_t)1 << 24;  // as the scan's dim; also the largest row stride
constexpr double kMaxThreads = 4294967295.0;      // of a launch

bool dtype_ok(int t) { return t == SSS_F32 || t == SSS_BF16; }
int64_t dtype_size(int t) { return t == SSS_BF16 ? 2 : 4; }
bool stride_ok(int64_t stride, int64_t dim) { return stride >= dim && stride <= kMaxRowDim; }
int status_of(hipError_t e) { return e == hipSuccess ? SSS_OK : SSS_ERR_HIP; }

int conv_impl(const void* x, int64_t x_stride, const float* weight, const float* bias, void* conv_state,
              const int32_t* cu_seqlens, const int32_t* state_indices, const uint8_t* has_initial, void* out,
              int64_t tokens, int64_t nseq, int64_t slots, int64_t dim, int64_t width, int io_dtype, int apply_silu,
              bool step, sss_stream_t stream) {
  if (!x || !weight || !out || (step ? !conv_state && width != 1 : !cu_seqlens)) return SSS_ERR_NULL_ARG;
  if (tokens < 0 || nseq < 0 || slots < 0 || dim < 1 || tokens > kMaxTokens || nseq > kMaxTokens ||
      slots > kMaxTokens || dim > kMaxRowDim ||
      (conv_state && (slots < 1 || (!state_indices && nseq > slots))))
    return SSS_ERR_BAD_DIM;
  if (width < 1 || width > 8 || !dtype_ok(io_dtype)) return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim)) return SSS_ERR_BAD_DIM;
  // threads of the launch: 256 per row and 512 channels, or 64 per 8 tokens and 128 channels
  const double threads = step ? (double)tokens * (double)((dim + 511) / 512) * 256.0
                              : (double)(tokens / 8 + 1) * (double)((dim + 127) / 128) * 64.0;
  if (threads > 2147483647.0) return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype);
  Regions r;
  r.in(x, span(tokens, x_stride, dim, es), es);
  r.in(weight, dim * width * 4, 4);
  r.in(bias, dim * 4, 4);
  r.in(cu_seqlens, (nseq + 1) * 4, 4);
  r.in(state_indices, nseq * 4, 4);
  r.in(has_initial, nseq, 1);
  r.output(conv_state, slots * (width - 1) * dim * es, es);
  r.output(out, tokens * dim * es, es);
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (tokens == 0 || nseq == 0) return SSS_OK;
  if (current_device_cus() <= 0) return SSS_ERR_HIP;
  PackedConvArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.w = weight;
  a.bias = bias;
  a.state = width > 1 ? conv_state : nullptr;  // one tap: nothing to keep
  a.cu = cu_seqlens;
  a.sidx = state_indices;
  a.init = has_initial;
  a.out = out;
  a.tokens = tokens;
  a.nseq = nseq;
  a.slots = width > 1 ? slots : 0;
  a.dim = dim;
  a.width = (int)width;
  a.bf16 = io_dtype == SSS_BF16;
  a.silu = apply_silu != 0;
  a.step = step;
  return status_of(launch_packed_conv(a, reinterpret_cast<hipStream_t>(stream)));
}

bool conv_bwd_dims_ok(int64_t batch, int64_t seqlen, int64_t dim, int64_t width) {
  return batch >= 1 && seqlen >= 1 && dim >= 1 && width >= 1 && width <= 8 && batch <= kMaxTokens &&
         seqlen <= kMaxTokens && dim <= kMaxRowDim &&
         (double)batch * (double)seqlen * (double)((dim + 63) / 64) <= (double)((int64_t)1 << 36);
}

int scan_dims(int64_t tokens, int64_t nseq, int64_t slots, int64_t dim, int64_t dstate) {
  if (tokens < 0 || nseq < 0 || slots < 0 || dim < 1 || dstate < 1 || tokens > kMaxTokens || nseq > kMaxTokens ||
      slots > kMaxTokens || dim > kMaxRowDim)
    return SSS_ERR_BAD_DIM;
  if (dstate > 64 || (dstate & (dstate - 1)) != 0) return SSS_ERR_UNSUPPORTED;
  if (dim * dstate > ((int64_t)1 << 30)) return SSS_ERR_BAD_DIM;
  if ((double)tokens * (double)dim > 1.8e18) return SSS_ERR_BAD_DIM;
  return SSS_OK;
}

int scan_impl(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride, const float* A, const void* B,
              int64_t b_stride, const void* C, int64_t c_stride, const float* D_skip, const void* z, int64_t z_stride,
              const float* delta_bias, unsigned flags, float* state, const int32_t* cu_seqlens,
              const int32_t* state_indices, const uint8_t* has_initial, void* y, int64_t tokens, int64_t nseq,
              int64_t slots, int64_t dim, int64_t dstate, int io_dtype, int bc_dtype, int y_dtype, void* workspace,
              size_t workspace_bytes, bool step, sss_stream_t stream) {
  if (!x || !delta || !A || !B || !C || !y || (step ? !state : !cu_seqlens)) return SSS_ERR_NULL_ARG;
  const int st = scan_dims(tokens, nseq, slots, dim, dstate);
  if (st != SSS_OK) return st;
  if (state && (slots < 1 || (!state_indices && nseq > slots))) return SSS_ERR_BAD_DIM;
  if (step && slot_update_threads(tokens, dim, dstate) > kMaxThreads) return SSS_ERR_BAD_DIM;
  if (!dtype_ok(io_dtype) || !dtype_ok(bc_dtype) || !dtype_ok(y_dtype)) return SSS_ERR_UNSUPPORTED;
  if ((flags & ~(unsigned)SSS_DELTA_SOFTPLUS) != 0) return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim) || !stride_ok(delta_stride, dim) || (z && !stride_ok(z_stride, dim)) ||
      !stride_ok(b_stride, dstate) || !stride_ok(c_stride, dstate))
    return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), bs = dtype_size(bc_dtype), ys = dtype_size(y_dtype);
  Regions r;
  r.in(x, span(tokens, x_stride, dim, es), es);
  r.in(delta, span(tokens, delta_stride, dim, es), es);
  r.in(A, dim * dstate * 4, 4);
  r.in(B, span(tokens, b_stride, dstate, bs), bs);
  r.in(C, span(tokens, c_stride, dstate, bs), bs);
  r.in(D_skip, dim * 4, 4);
  r.in(z, span(tokens, z_stride, dim, es), es);
  r.in(delta_bias, dim * 4, 4);
  r.in(cu_seqlens, (nseq + 1) * 4, 4);
  r.in(state_indices, nseq * 4, 4);
  r.in(has_initial, nseq, 1);
  r.output(state, slots * dim * dstate * 4, 4);
  r.output(y, tokens * dim * ys, ys);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (tokens == 0 || nseq == 0) return SSS_OK;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  PackedScanArgs a{};
  a.x = x;
  a.delta = delta;
  a.A = A;
  a.B = B;
  a.C = C;
  a.Dsk = D_skip;
  a.z = z;
  a.delta_bias = delta_bias;
  a.state = state;
  a.cu = cu_seqlens;
  a.sidx = state_indices;
  a.init = has_initial;
  a.y = y;
  a.sx = x_stride;
  a.sd = delta_stride;
  a.sz = z ? z_stride : 0;
  a.sb = b_stride;
  a.sc = c_stride;
  a.tokens = tokens;
  a.nseq = nseq;
  a.slots = slots;
  a.dim = dim;
  a.dstate = (int)dstate;
  a.bf16 = io_dtype == SSS_BF16;
  a.bc_bf16 = bc_dtype == SSS_BF16;
  a.y_bf16 = y_dtype == SSS_BF16;
  a.softplus = (flags & SSS_DELTA_SOFTPLUS) != 0;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (step) return status_of(launch_slot_update(a, s));
  const PackedScanPlan pl = plan_packed_scan(tokens, dim, dstate, cus);
  if ((double)pl.chunks * (double)((dim + 63) / 64) > (double)((int64_t)1 << 24)) return SSS_ERR_BAD_DIM;
  if (pl.ws_total > 0) {
    if (workspace == nullptr || workspace_bytes < pl.ws_total) return SSS_ERR_WORKSPACE;
    r.output(workspace, (int64_t)pl.ws_total, 16);
    if (!r.ok()) return SSS_ERR_ALIAS;
  }
  a.workspace = workspace;
  if (env_int("SSS_LOG", 0))
    std::fprintf(stderr, "[sss] selective_scan_packed_fwd T=%lld seqs=%lld D=%lld N=%lld %s: chunks=%d of %lld ws=%zu\n",
                 (long long)tokens, (long long)nseq, (long long)dim, (long long)dstate,
                 io_dtype == SSS_BF16 ? "bf16" : "f32", pl.chunks, (long long)pl.K, pl.ws_total);
  return status_of(launch_packed_scan(a, pl, s));
}

// rows of a norm: norm_lanes threads for each row and group, in workgroups of at most 1024
int norm_dims(int64_t rows, int64_t dim, int64_t group, bool fp32) {
  if (rows < 0 || dim < 1 || group < 1 || rows > kMaxTokens || dim > kMaxRowDim || dim % group != 0)
    return SSS_ERR_BAD_DIM;
  if (group > kMaxNormDim) return SSS_ERR_UNSUPPORTED;
  if ((double)rows * (double)(dim / group) * (double)norm_lanes(group, fp32) + 1024.0 > kMaxThreads) return SSS_ERR_BAD_DIM;
  return SSS_OK;
}

// its gradients: each group a workgroup at least (and otherwise no more than four per CU)
int norm_bwd_dims(int64_t rows, int64_t dim, int64_t group, bool fp32) {
  const int st = norm_dims(rows, dim, group, fp32);
  if (st == SSS_OK && (double)(dim / group) * (double)std::max(256, norm_lanes(group, fp32)) > kMaxThreads)
    return SSS_ERR_BAD_DIM;
  return st;
}

// bytes for either kernel shape: a query does not know the types
size_t norm_bwd_bytes(int64_t rows, int64_t dim, int64_t group, int vectors, int device) {
  int cus = device_cus(device);
  if (cus <= 0) cus = 256;
  size_t most = 0;
  for (const bool fp32 : {false, true})
    if (norm_bwd_dims(rows, dim, group, fp32) == SSS_OK)
      most = std::max(most, plan_norm_bwd(rows, group, dim / group, vectors, fp32, cus).ws_total);
  return most;
}

}  // namespace

extern "C" {

int rms_norm_gated_fwd(const void* x, int64_t x_stride, const float* weight, const void* z, int64_t z_stride, void* out,
                       float* rstd, int64_t rows, int64_t dim, int64_t group, float eps, unsigned flags, int x_dtype,
                       int out_dtype, sss_stream_t stream) {
  if (!x || !weight || !out) return SSS_ERR_NULL_ARG;
  const bool fp32 = x_dtype == SSS_F32 || out_dtype == SSS_F32;
  const int st = norm_dims(rows, dim, group, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || (flags & ~(unsigned)SSS_NORM_BEFORE_GATE) != 0)
    return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim) || (z && !stride_ok(z_stride, dim))) return SSS_ERR_BAD_DIM;
  const int64_t xs = dtype_size(x_dtype), os = dtype_size(out_dtype);
  Regions r;
  r.in(x, span(rows, x_stride, dim, xs), xs);
  r.in(weight, dim * 4, 4);
  r.in(z, span(rows, z_stride, dim, os), os);
  r.output(out, rows * dim * os, os);
  r.output(rstd, rows * (dim / group) * 4, 4);
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (rows == 0) return SSS_OK;
  GatedNormArgs a{};
  a.x = x;
  a.z = z;
  a.w = weight;
  a.out = out;
  a.rstd = rstd;
  a.rows = rows;
  a.group = group;
  a.groups = dim / group;
  a.sx = x_stride;
  a.sz = z ? z_stride : 0;
  a.eps = eps;
  a.x_bf16 = x_dtype == SSS_BF16;
  a.z_bf16 = out_dtype == SSS_BF16;
  a.norm_first = (flags & SSS_NORM_BEFORE_GATE) != 0;
  return status_of(launch_gated_norm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t rms_norm_gated_bwd_workspace_size(int64_t rows, int64_t dim, int64_t group, int device) {
  return norm_bwd_bytes(rows, dim, group, 1, device);
}

int rms_norm_gated_bwd(const void* dout, const void* x, int64_t x_stride, const float* weight, const void* z,
                       int64_t z_stride, const float* rstd, void* dx, void* dz, int64_t dz_stride, float* dweight,
                       int64_t rows, int64_t dim, int64_t group, unsigned flags, int x_dtype, int out_dtype,
                       void* workspace, size_t workspace_bytes, sss_stream_t stream) {
  if (!dweight || (rows != 0 && (!dout || !x || !weight || !rstd || !dx || (z && !dz)))) return SSS_ERR_NULL_ARG;
  const bool fp32 = x_dtype == SSS_F32 || out_dtype == SSS_F32;
  const int st = norm_bwd_dims(rows, dim, group, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || (flags & ~(unsigned)SSS_NORM_BEFORE_GATE) != 0)
    return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim) || (z && (!stride_ok(z_stride, dim) || !stride_ok(dz_stride, dim))))
    return SSS_ERR_BAD_DIM;
  const int64_t xs = dtype_size(x_dtype), os = dtype_size(out_dtype);
  Regions r;
  r.in(dout, rows * dim * os, os);
  r.in(x, span(rows, x_stride, dim, xs), xs);
  r.in(weight, dim * 4, 4);
  r.in(z, span(rows, z_stride, dim, os), os);
  r.in(rstd, rows * (dim / group) * 4, 4);
  r.output(dx, rows * dim * xs, xs);
  r.output(z ? dz : nullptr, span(rows, dz_stride, dim, os), os);
  r.output(dweight, dim * 4, 4);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const NormPlan pl = plan_norm_bwd(rows, group, dim / group, 1, fp32, cus);
  if (workspace == nullptr || workspace_bytes < pl.ws_total) return SSS_ERR_WORKSPACE;
  r.output(workspace, (int64_t)pl.ws_total, 16);
  if (!r.ok()) return SSS_ERR_ALIAS;
  GatedNormArgs a{};
  a.x = x;
  a.z = z;
  a.w = weight;
  a.rstd = const_cast<float*>(rstd);
  a.dout = dout;
  a.dx = dx;
  a.dz = z ? dz : nullptr;
  a.dw = dweight;
  a.workspace = workspace;
  a.rows = rows;
  a.group = group;
  a.groups = dim / group;
  a.sx = x_stride;
  a.sz = z ? z_stride : 0;
  a.sdz = z ? dz_stride : 0;
  a.x_bf16 = x_dtype == SSS_BF16;
  a.z_bf16 = out_dtype == SSS_BF16;
  a.norm_first = (flags & SSS_NORM_BEFORE_GATE) != 0;
  return status_of(launch_gated_norm_bwd(a, pl, reinterpret_cast<hipStream_t>(stream)));
}

int rms_norm_residual_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          const float* post_weight, const float* scale, const float* weight, void* out,
                          void* residual_out, float* rstd_post, float* rstd, int64_t rows, int64_t dim, float alpha,
                          float eps, int io_dtype, int residual_dtype, sss_stream_t stream) {
  if (!x || !weight || !out || !residual_out) return SSS_ERR_NULL_ARG;
  const bool fp32 = io_dtype == SSS_F32 || residual_dtype == SSS_F32;
  const int st = norm_dims(rows, dim, dim, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(io_dtype) || !dtype_ok(residual_dtype)) return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim) || (residual && !stride_ok(residual_stride, dim))) return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), hs = dtype_size(residual_dtype);
  // the residual stream may be updated in place: the same rows, or no shared memory at all
  const bool in_place = residual == residual_out && (residual_stride == dim || rows <= 1);
  Regions r;
  r.in(x, span(rows, x_stride, dim, es), es);
  if (!in_place) r.in(residual, span(rows, residual_stride, dim, hs), hs);
  r.in(post_weight, dim * 4, 4);
  r.in(scale, dim * 4, 4);
  r.in(weight, dim * 4, 4);
  r.output(out, rows * dim * es, es);
  r.output(residual_out, rows * dim * hs, hs);
  r.output(post_weight ? rstd_post : nullptr, rows * 4, 4);
  r.output(rstd, rows * 4, 4);
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (rows == 0) return SSS_OK;
  ResNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.wp = post_weight;
  a.scale = scale;
  a.w = weight;
  a.out = out;
  a.residual_out = residual_out;
  a.rstd_post = rstd_post;
  a.rstd = rstd;
  a.rows = rows;
  a.dim = dim;
  a.sx = x_stride;
  a.sr = residual ? residual_stride : 0;
  a.eps = eps;
  a.alpha = alpha;
  a.x_bf16 = io_dtype == SSS_BF16;
  a.h_bf16 = residual_dtype == SSS_BF16;
  return status_of(launch_res_norm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t rms_norm_residual_bwd_workspace_size(int64_t rows, int64_t dim, int device) {
  return norm_bwd_bytes(rows, dim, dim, 3, device);
}

int rms_norm_residual_bwd(const void* dout, const void* dresidual_out, const void* x, int64_t x_stride,
                          const void* residual_out, const float* post_weight, const float* scale, const float* weight,
                          const float* rstd_post, const float* rstd, void* dx, void* dresidual, float* dweight,
                          float* dpost_weight, float* dscale, int64_t rows, int64_t dim, float alpha, int io_dtype,
                          int residual_dtype, void* workspace, size_t workspace_bytes, sss_stream_t stream) {
  if (!dweight || (post_weight && !dpost_weight) || (scale && !dscale)) return SSS_ERR_NULL_ARG;
  if (rows != 0 && (!dout || !residual_out || !weight || !rstd || !dx || (post_weight && !rstd_post) ||
                    ((post_weight || scale) && !x)))
    return SSS_ERR_NULL_ARG;
  const bool fp32 = io_dtype == SSS_F32 || residual_dtype == SSS_F32;
  const int st = norm_bwd_dims(rows, dim, dim, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(io_dtype) || !dtype_ok(residual_dtype)) return SSS_ERR_UNSUPPORTED;
  if (x && !stride_ok(x_stride, dim)) return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), hs = dtype_size(residual_dtype);
  Regions r;
  r.in(dout, rows * dim * es, es);
  r.in(dresidual_out, rows * dim * hs, hs);
  r.in(x, span(rows, x_stride, dim, es), es);
  r.in(residual_out, rows * dim * hs, hs);
  r.in(post_weight, dim * 4, 4);
  r.in(scale, dim * 4, 4);
  r.in(weight, dim * 4, 4);
  r.in(post_weight ? rstd_post : nullptr, rows * 4, 4);
  r.in(rstd, rows * 4, 4);
  r.output(dx, rows * dim * es, es);
  r.output(dresidual, rows * dim * hs, hs);
  r.output(dweight, dim * 4, 4);
  r.output(post_weight ? dpost_weight : nullptr, dim * 4, 4);
  r.output(scale ? dscale : nullptr, dim * 4, 4);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const NormPlan pl = plan_norm_bwd(rows, dim, 1, 3, fp32, cus);
  if (workspace == nullptr || workspace_bytes < pl.ws_total) return SSS_ERR_WORKSPACE;
  r.output(workspace, (int64_t)pl.ws_total, 16);
  if (!r.ok()) return SSS_ERR_ALIAS;
  ResNormArgs a{};
  a.x = x;
  a.wp = post_weight;
  a.scale = scale;
  a.w = weight;
  a.residual_out = const_cast<void*>(residual_out);
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd = const_cast<float*>(rstd);
  a.dout = dout;
  a.dres_out = dresidual_out;
  a.dx = dx;
  a.dres = dresidual;
  a.dw = dweight;
  a.dwp = dpost_weight;
  a.dscale = dscale;
  a.workspace = workspace;
  a.rows = rows;
  a.dim = dim;
  a.sx = x ? x_stride : 0;
  a.alpha = alpha;
  a.x_bf16 = io_dtype == SSS_BF16;
  a.h_bf16 = residual_dtype == SSS_BF16;
  return status_of(launch_res_norm_bwd(a, pl, reinterpret_cast<hipStream_t>(stream)));
}

int causal_conv1d_packed_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias, void* conv_state,
                             const int32_t* cu_seqlens, const int32_t* state_indices, const uint8_t* has_initial,
                             void* out, int64_t tokens, int64_t nseq, int64_t slots, int64_t dim, int64_t width,
                             int io_dtype, int apply_silu, sss_stream_t stream) {
  return conv_impl(x, x_stride, weight, bias, conv_state, cu_seqlens, state_indices, has_initial, out, tokens, nseq,
                   slots, dim, width, io_dtype, apply_silu, false, stream);
}

int causal_conv1d_update(const void* x, int64_t x_stride, const float* weight, const float* bias, void* conv_state,
                         const int32_t* state_indices, void* out, int64_t batch, int64_t slots, int64_t dim,
                         int64_t width, int io_dtype, int apply_silu, sss_stream_t stream) {
  return conv_impl(x, x_stride, weight, bias, conv_state, nullptr, state_indices, nullptr, out, batch, batch, slots,
                   dim, width, io_dtype, apply_silu, true, stream);
}

size_t causal_conv1d_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype,
                                        int device) {
  if (!conv_bwd_dims_ok(batch, seqlen, dim, width) || !dtype_ok(io_dtype)) return 0;
  int cus = device_cus(device);
  if (cus <= 0) cus = 256;
  return plan_conv_bwd(batch, seqlen, dim, width, io_dtype == SSS_BF16, cus).ws_total;
}

int causal_conv1d_bwd(const void* x, int64_t x_batch_stride, int64_t x_stride, const float* weight, const float* bias,
                      const void* dout, void* dx, int64_t dx_batch_stride, int64_t dx_stride, float* dweight,
                      float* dbias, int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype,
                      int dout_dtype, int dx_dtype, int apply_silu, void* workspace, size_t workspace_bytes,
                      sss_stream_t stream) {
  if (!x || !weight || !dout || !dx || !dweight || (bias && !dbias)) return SSS_ERR_NULL_ARG;
  if (width < 1 || width > 8) return batch < 1 || seqlen < 1 || dim < 1 ? SSS_ERR_BAD_DIM : SSS_ERR_UNSUPPORTED;
  if (!conv_bwd_dims_ok(batch, seqlen, dim, width)) return SSS_ERR_BAD_DIM;
  // each of the gradients in fp32 or in x's type
  if (!dtype_ok(io_dtype) || (dout_dtype != SSS_F32 && dout_dtype != io_dtype) ||
      (dx_dtype != SSS_F32 && dx_dtype != io_dtype))
    return SSS_ERR_UNSUPPORTED;
  const int64_t kMaxBatchStride = (int64_t)1 << 46;
  if (!stride_ok(x_stride, dim) || !stride_ok(dx_stride, dim) || x_batch_stride < 0 || dx_batch_stride < 0 ||
      x_batch_stride > kMaxBatchStride || dx_batch_stride > kMaxBatchStride)
    return SSS_ERR_BAD_DIM;
  // rows of dx may not share elements: one batch entry after the other, or (time-major) one step after
  // the other with the batch entries inside it
  if (batch > 1 && dx_batch_stride < (seqlen - 1) * dx_stride + dim &&
      !(dx_batch_stride >= dim && (seqlen == 1 || dx_stride >= (batch - 1) * dx_batch_stride + dim)))
    return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), dos = dtype_size(dout_dtype), dxs = dtype_size(dx_dtype);
  Regions r;
  r.in(x, (batch - 1) * x_batch_stride * es + span(seqlen, x_stride, dim, es), es);
  r.in(weight, dim * width * 4, 4);
  r.in(bias, dim * 4, 4);
  r.in(dout, batch * seqlen * dim * dos, dos);
  r.output(dx, (batch - 1) * dx_batch_stride * dxs + span(seqlen, dx_stride, dim, dxs), dxs);
  r.output(dweight, dim * width * 4, 4);
  r.output(bias ? dbias : nullptr, dim * 4, 4);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const ConvBwdPlan pl = plan_conv_bwd(batch, seqlen, dim, width, io_dtype == SSS_BF16, cus);
  if ((double)pl.segments * (double)batch * (double)((dim + 63) / 64) > (double)((int64_t)1 << 24) * 2) return SSS_ERR_BAD_DIM;
  if (workspace == nullptr || workspace_bytes < pl.ws_total) return SSS_ERR_WORKSPACE;
  r.output(workspace, (int64_t)pl.ws_total, 16);
  if (!r.ok()) return SSS_ERR_ALIAS;
  ConvBwdArgs a{};
  a.x = x;
  a.x_row = x_stride;
  a.x_batch = x_batch_stride;
  a.w = weight;
  a.bias = bias;
  a.dout = dout;
  a.dx = dx;
  a.dx_row = dx_stride;
  a.dx_batch = dx_batch_stride;
  a.dw = dweight;
  a.db = bias ? dbias : nullptr;
  a.workspace = workspace;
  a.batch = batch;
  a.seqlen = seqlen;
  a.dim = dim;
  a.width = (int)width;
  a.bf16 = io_dtype == SSS_BF16;
  a.dout_bf16 = dout_dtype == SSS_BF16;
  a.dx_bf16 = dx_dtype == SSS_BF16;
  a.silu = apply_silu != 0;
  return status_of(launch_conv_bwd(a, pl, reinterpret_cast<hipStream_t>(stream)));
}

size_t selective_scan_packed_fwd_workspace_size(int64_t tokens, int64_t dim, int64_t dstate, int device) {
  if (scan_dims(tokens, 0, 0, dim, dstate) != SSS_OK || tokens < 1) return 0;
  int cus = device_cus(device);
  if (cus <= 0) cus = 256;
  return plan_packed_scan(tokens, dim, dstate, cus).ws_total;
}

int selective_scan_packed_fwd(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride, const float* A,
                              const void* B, int64_t b_stride, const void* C, int64_t c_stride, const float* D_skip,
                              const void* z, int64_t z_stride, const float* delta_bias, unsigned flags, float* state,
                              const int32_t* cu_seqlens, const int32_t* state_indices, const uint8_t* has_initial,
                              void* y, int64_t tokens, int64_t nseq, int64_t slots, int64_t dim, int64_t dstate,
                              int io_dtype, int bc_dtype, int y_dtype, void* workspace, size_t workspace_bytes,
                              sss_stream_t stream) {
  return scan_impl(x, x_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D_skip, z, z_stride, delta_bias,
                   flags, state, cu_seqlens, state_indices, has_initial, y, tokens, nseq, slots, dim, dstate, io_dtype,
                   bc_dtype, y_dtype, workspace, workspace_bytes, false, stream);
}

int selective_state_update_slots(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride,
                                 const float* A, const void* B, int64_t b_stride, const void* C, int64_t c_stride,
                                 const float* D_skip, const void* z, int64_t z_stride, const float* delta_bias,
                                 unsigned flags, float* state, const int32_t* state_indices, void* y, int64_t batch,
                                 int64_t slots, int64_t dim, int64_t dstate, int io_dtype, int bc_dtype, int y_dtype,
                                 sss_stream_t stream) {
  return scan_impl(x, x_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D_skip, z, z_stride, delta_bias,
                   flags, state, nullptr, state_indices, nullptr, y, batch, batch, slots, dim, dstate, io_dtype,
                   bc_dtype, y_dtype, nullptr, 0, true, stream);
}

int layer_norm_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const float* weight,
                   const float* bias, void* out, void* residual_out, float* mean, float* rstd, int64_t rows, int64_t dim,
                   int64_t group, float eps, int io_dtype, int residual_dtype, sss_stream_t stream) {
  if (!x || !out) return SSS_ERR_NULL_ARG;
  const bool stream_used = residual || residual_out;
  const int hd = stream_used ? residual_dtype : io_dtype;
  const bool fp32 = io_dtype == SSS_F32 || hd == SSS_F32;
  const int st = norm_dims(rows, dim, group, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(io_dtype) || !dtype_ok(hd)) return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim) || (residual && !stride_ok(residual_stride, dim))) return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), hs = dtype_size(hd);
  // the residual stream may be updated in place: the same rows, or no shared memory at all
  const bool in_place = residual && residual == residual_out && (residual_stride == dim || rows <= 1);
  Regions r;
  r.in(x, span(rows, x_stride, dim, es), es);
  if (!in_place) r.in(residual, span(rows, residual_stride, dim, hs), hs);
  r.in(weight, dim * 4, 4);
  r.in(bias, dim * 4, 4);
  r.output(out, rows * dim * es, es);
  r.output(residual_out, rows * dim * hs, hs);
  r.output(mean, rows * (dim / group) * 4, 4);
  r.output(rstd, rows * (dim / group) * 4, 4);
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (rows == 0) return SSS_OK;
  LayerNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.w = weight;
  a.b = bias;
  a.out = out;
  a.residual_out = residual_out;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.group = group;
  a.groups = dim / group;
  a.sx = x_stride;
  a.sr = residual ? residual_stride : 0;
  a.eps = eps;
  a.x_bf16 = io_dtype == SSS_BF16;
  a.h_bf16 = hd == SSS_BF16;
  return status_of(launch_layer_norm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t layer_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t group, int device) {
  return norm_bwd_bytes(rows, dim, group, 2, device);
}

int layer_norm_bwd(const void* dout, const void* dresidual_out, const void* x, int64_t x_stride, const float* weight,
                   const float* mean, const float* rstd, void* dx, void* dresidual, float* dweight, float* dbias,
                   int64_t rows, int64_t dim, int64_t group, int io_dtype, int x_dtype, void* workspace,
                   size_t workspace_bytes, sss_stream_t stream) {
  if ((rows != 0 && (!dout || !x || !mean || !rstd || !dx)) || (weight && !dweight)) return SSS_ERR_NULL_ARG;
  const bool fp32 = io_dtype == SSS_F32 || x_dtype == SSS_F32;
  const int st = norm_bwd_dims(rows, dim, group, fp32);
  if (st != SSS_OK) return st;
  if (!dtype_ok(io_dtype) || !dtype_ok(x_dtype)) return SSS_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, dim)) return SSS_ERR_BAD_DIM;
  const int64_t es = dtype_size(io_dtype), hs = dtype_size(x_dtype);
  Regions r;
  r.in(dout, rows * dim * es, es);
  r.in(dresidual_out, rows * dim * hs, hs);
  r.in(x, span(rows, x_stride, dim, hs), hs);
  r.in(weight, dim * 4, 4);
  r.in(mean, rows * (dim / group) * 4, 4);
  r.in(rstd, rows * (dim / group) * 4, 4);
  r.output(dx, rows * dim * es, es);
  r.output(dresidual, rows * dim * hs, hs);
  r.output(dweight, dim * 4, 4);
  r.output(dbias, dim * 4, 4);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const NormPlan pl = plan_norm_bwd(rows, group, dim / group, (dweight ? 1 : 0) + (dbias ? 1 : 0), fp32, cus);
  if (pl.ws_total > 0) {
    if (workspace == nullptr || workspace_bytes < pl.ws_total) return SSS_ERR_WORKSPACE;
    r.output(workspace, (int64_t)pl.ws_total, 16);
    if (!r.ok()) return SSS_ERR_ALIAS;
  }
  LayerNormArgs a{};
  a.x = x;
  a.w = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dout = dout;
  a.dres_out = dresidual_out;
  a.dx = dx;
  a.dres = dresidual;
  a.dw = dweight;
  a.db = dbias;
  a.workspace = workspace;
  a.rows = rows;
  a.group = group;
  a.groups = dim / group;
  a.sx = x_stride;
  a.x_bf16 = io_dtype == SSS_BF16;
  a.h_bf16 = x_dtype == SSS_BF16;
  return status_of(launch_layer_norm_bwd(a, pl, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

// conv_bwd.hip -- gfx950 kernels of the causal depthwise convolution's gradients.
//
// With v[t] = bias + sum_{k<W} w[k] x[t-(W-1)+k] per channel, out = silu(v) or v, and the
// gradient dout of out:
//   dv[t]  = dout[t] * silu'(v[t])       (silu'(v) = s (1 + v (1 - s)), s = 1 / (1 + e^-v))
//   dx[u]  = sum_k w[k] dv[u + (W-1) - k]   (terms past the sequence's end are zero)
//   dw[k]  = sum_{b,t} dv[t] x[t-(W-1)+k],  dbias = sum_{b,t} dv[t].
// v is recomputed from x, so that nothing of the forward call is kept.  Streaming: x and dout
// in, dx out.
#include "vec.h"
#include "kernels.h"

#include <algorithm>

namespace sss {

constexpr int kCBwdU = 4;  // steps per load batch

struct CBwdGeo {
  int64_t x_row, x_batch, dx_row, dx_batch;  // strides in elements
  int L, D, seg_len, S, batch, ngroups;
  int dx_bf16;
};

// One wave = 64 lanes x CPL adjacent channels, one batch row and one time segment.  It walks
// its steps and the W-1 after them (the next segment's, whose dv its last dx need), with the
// last W inputs and the W unfinished dx of each channel in registers; dw and dbias are summed
// over the segment's own steps and leave as one partial per segment.
template <int W, bool BF16, bool DOBF16, int CPL>
__global__ __launch_bounds__(64) void conv_bwd_kernel(const char* __restrict__ x, const float* __restrict__ w,
                                                      const float* __restrict__ bias, const char* __restrict__ dout,
                                                      char* __restrict__ dx, float* __restrict__ part, CBwdGeo g,
                                                      int apply_silu) {
  using RX = Vec<BF16, CPL>;
  using RD = Vec<DOBF16, CPL>;
  constexpr int ES = RX::ES, DS = RD::ES;
  const int lane = threadIdx.x;
  uint32_t lid = xcd_remap(blockIdx.x, gridDim.x);
  const int grp = (int)(lid % (uint32_t)g.ngroups);
  lid /= (uint32_t)g.ngroups;
  const int b = (int)(lid % (uint32_t)g.batch);
  const int s = (int)(lid / (uint32_t)g.batch);
  const int dl = grp * 64 * CPL + lane * CPL;
  const int dc = min(dl, g.D - CPL);
  const int skip = min(dl - dc, CPL);  // channels that a lane before has: not stored here
  const int tb = s * g.seg_len;
  const int te = min(tb + g.seg_len, g.L);
  const int64_t D = g.D;

  float wk[CPL][W], bv[CPL], dw[CPL][W], db[CPL], win[CPL][W], acc[CPL][W];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      wk[c][k] = w[(int64_t)(dc + c) * W + k];
      dw[c][k] = 0.0f;
      acc[c][k] = 0.0f;
    }
    bv[c] = bias != nullptr ? bias[dc + c] : 0.0f;
    db[c] = 0.0f;
  }
  const int64_t xrow = g.x_row * ES, drow = D * DS;
  const char* const xl = x + ((int64_t)b * g.x_batch + dc) * ES;
  const char* const dl_ = dout + ((int64_t)b * g.L * D + dc) * DS;
  const int xs = g.dx_bf16 ? 2 : 4;
  const int64_t dxrow = g.dx_row * xs;
  char* const ol = dx + ((int64_t)b * g.dx_batch + dc) * xs;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = tb - (W - 1) + k;
    RX r;
    if (t >= 0) r.load(xl + (int64_t)t * xrow);
    else r.zero();
#pragma unroll
    for (int c = 0; c < CPL; ++c) win[c][k] = r.get(c);
  }

  RX xq[2][kCBwdU];
  RD dq[2][kCBwdU];
  const int last = g.L - 1;
  auto load = [&](int slot, int t0) {
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i) {
      const int t = min(t0 + i, last);
      xq[slot][i].template load<true>(xl + (int64_t)t * xrow);
      dq[slot][i].template load<true>(dl_ + (int64_t)t * drow);
    }
  };
  // step t; acc[c][k] is the unfinished dx of row t-(W-1)+k
  auto step = [&](const RX& xr, const RD& dr, int t) {
    float o[CPL];
    const bool inside = t <= last, own = t < te;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      win[c][W - 1] = xr.get(c);
      float dv = inside ? dr.get(c) : 0.0f;
      if (apply_silu) {
        float v = bv[c];
#pragma unroll
        for (int k = 0; k < W; ++k) v = __builtin_fmaf(wk[c][k], win[c][k], v);
        const float sg = fast_rcp(1.0f + fast_exp2(-v * kLog2e));
        dv *= sg * __builtin_fmaf(v, 1.0f - sg, 1.0f);
      }
#pragma unroll
      for (int k = 0; k < W; ++k) acc[c][k] = __builtin_fmaf(wk[c][k], dv, acc[c][k]);
      const float dvo = own ? dv : 0.0f;
      db[c] += dvo;
#pragma unroll
      for (int k = 0; k < W; ++k) dw[c][k] = __builtin_fmaf(dvo, win[c][k], dw[c][k]);
      o[c] = acc[c][0];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        acc[c][k] = acc[c][k + 1];
        win[c][k] = win[c][k + 1];
      }
      acc[c][W - 1] = 0.0f;
    }
    const int u = t - (W - 1);
    if (u >= tb) {
      char* const p = ol + (int64_t)u * dxrow;
      if (g.dx_bf16) {
        Vec<true, CPL> r;
        r.set(o);
        r.template store_from<true>(p, skip);
      } else {
        Vec<false, CPL> r;
        r.set(o);
        r.template store_from<true>(p, skip);
      }
    }
  };
  const int tl = te + W - 1;  // one past the last step walked
  load(0, tb);
  int t0 = tb;
  for (; t0 + 2 * kCBwdU <= tl; t0 += 2 * kCBwdU) {
    load(1, t0 + kCBwdU);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i) step(xq[0][i], dq[0][i], t0 + i);
    load(0, t0 + 2 * kCBwdU);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i) step(xq[1][i], dq[1][i], t0 + kCBwdU + i);
  }
  if (t0 < tl) {
    load(1, t0 + kCBwdU);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i)
      if (t0 + i < tl) step(xq[0][i], dq[0][i], t0 + i);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i)
      if (t0 + kCBwdU + i < tl) step(xq[1][i], dq[1][i], t0 + kCBwdU + i);
  }
  // partial sums [s][b][W + 1][D]: the taps, then the bias
  float* const pp = part + ((int64_t)s * g.batch + b) * (W + 1) * D + dc;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    float v[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) v[c] = k < W ? dw[c][k < W ? k : 0] : db[c];
    Vec<false, CPL> r;
    r.set(v);
    r.store_from(pp + (int64_t)k * D, skip);
  }
}

// dweight (D, W) and dbias (D) from the partials, added in their order: 64 columns (a wave's
// lanes) and 4 row ranges per workgroup, the ranges joined in LDS.
static __global__ __launch_bounds__(256) void conv_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                                  float* __restrict__ db, int rows, int W, int D) {
  __shared__ float lds[256];
  const int64_t cols = (int64_t)(W + 1) * D;
  const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int64_t cc = min(col, cols - 1);
  const int part_id = threadIdx.x >> 6;
  const int per = (rows + 3) / 4;
  const int r1 = min(rows, (part_id + 1) * per);
  float s = 0.0f;
  for (int r = part_id * per; r < r1; r += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)min(r + i, r1 - 1) * cols + cc];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += r + i < r1 ? v[i] : 0.0f;
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x >= 64 || col >= cols) return;
  s = (lds[threadIdx.x] + lds[threadIdx.x + 64]) + (lds[threadIdx.x + 128] + lds[threadIdx.x + 192]);
  const int k = (int)(col / D);
  const int64_t d = col - (int64_t)k * D;
  if (k < W) dw[d * W + k] = s;
  else if (db != nullptr) db[d] = s;
}

ConvBwdPlan plan_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, bool bf16, int num_cus) {
  ConvBwdPlan pl{};
  const int wide = bf16 ? 4 : 2;
  pl.cpl = dim >= wide ? wide : 1;
  const int64_t waves = batch * ((dim + 64 * pl.cpl - 1) / (64 * pl.cpl));
  const int64_t target = (int64_t)std::max(num_cus, 1) * 16;
  int64_t S = waves >= target ? 1 : (target + waves - 1) / waves;
  // every segment walks width-1 steps of the next one again and leaves a partial: 64 steps at least
  S = std::min<int64_t>(S, std::max<int64_t>(1, seqlen / 64));
  const int forced = env_int("SSS_FORCE_SEGMENTS", 0);
  if (forced > 0) S = std::min<int64_t>(forced, seqlen);
  pl.seg_len = (seqlen + S - 1) / S;
  pl.segments = (int)((seqlen + pl.seg_len - 1) / pl.seg_len);
  pl.ws_total = (size_t)pl.segments * batch * (width + 1) * dim * 4;
  return pl;
}

template <int W, bool BF16, bool DOBF16, int CPL>
static hipError_t run_bwd(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  CBwdGeo g{};
  g.x_row = a.x_row;
  g.x_batch = a.x_batch;
  g.dx_row = a.dx_row;
  g.dx_batch = a.dx_batch;
  g.L = (int)a.seqlen;
  g.D = (int)a.dim;
  g.seg_len = (int)pl.seg_len;
  g.S = pl.segments;
  g.batch = (int)a.batch;
  g.ngroups = (int)((a.dim + 64 * CPL - 1) / (64 * CPL));
  g.dx_bf16 = a.dx_bf16;
  const int64_t grid = (int64_t)g.ngroups * a.batch * pl.segments;
  hipLaunchKernelGGL((conv_bwd_kernel<W, BF16, DOBF16, CPL>), dim3((unsigned)grid), dim3(64), 0, stream,
                     (const char*)a.x, a.w, a.bias, (const char*)a.dout, (char*)a.dx, (float*)a.workspace, g, a.silu);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t cols = (int64_t)(W + 1) * a.dim;
  hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, stream,
                     (const float*)a.workspace, a.dw, a.db, (int)(pl.segments * a.batch), W, (int)a.dim);
  return hipGetLastError();
}

template <int W>
static hipError_t run_bwd_types(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  if (a.bf16) {
    if (a.dout_bf16) return pl.cpl == 4 ? run_bwd<W, true, true, 4>(a, pl, stream) : run_bwd<W, true, true, 1>(a, pl, stream);
    return pl.cpl == 4 ? run_bwd<W, true, false, 4>(a, pl, stream) : run_bwd<W, true, false, 1>(a, pl, stream);
  }
  return pl.cpl == 2 ? run_bwd<W, false, false, 2>(a, pl, stream) : run_bwd<W, false, false, 1>(a, pl, stream);
}

hipError_t launch_conv_bwd(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  switch (a.width) {
    case 1: return run_bwd_types<1>(a, pl, stream);
    case 2: return run_bwd_types<2>(a, pl, stream);
    case 3: return run_bwd_types<3>(a, pl, stream);
    case 4: return run_bwd_types<4>(a, pl, stream);
    case 5: return run_bwd_types<5>(a, pl, stream);
    case 6: return run_bwd_types<6>(a, pl, stream);
    case 7: return run_bwd_types<7>(a, pl, stream);
    case 8: return run_bwd_types<8>(a, pl, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sss

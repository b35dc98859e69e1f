// conv_bwd.hip -- gfx950 kernels of the causal depthwise convolution's gradients.
//
// With v[t] = bias + sum_{k<W} w[k] x[t-(W-1)+k] per channel, out = silu(v) or v, and the
// gradient dout of out:
//   dv[t]  = dout[t] * silu'(v[t])       (silu'(v) = s (1 + v (1 - s)), s = 1 / (1 + e^-v))
//   dx[u]  = sum_k w[k] dv[u + (W-1) - k]   (terms past the sequence's end are zero)
//   dw[k]  = sum_{b,t} dv[t] x[t-(W-1)+k],  dbias = sum_{b,t} dv[t].
// v is recomputed from x, so that nothing of the forward call is kept.
//
// Bound by memory: x and dout in, dx out.  2 x 8192 x 5120 bf16 moves 512 MB (its partial sums
// among them) in 105-108 us, 4.8 TB/s, and the sums take 5 us; its VALU would take 59 us alone.
// Tiles that load all their rows at once without a walk read the W-1 rows before and after them
// again and measured 122-142 us.
#include "colsum.h"
#include "vec.h"
#include "kernels.h"

#include <algorithm>

namespace sss {

constexpr int kCBwdU = 4;  // steps per load batch

struct CBwdGeo {
  int64_t x_row, x_batch, dx_row, dx_batch;  // strides in elements
  int L, D, seg_len, batch, ngroups;
  int dx_bf16;
};

// One wave = 64 lanes x CPL adjacent channels, one batch row and one time segment.  It walks
// its steps and the W-1 after them (the next segment's, whose dv its last dx need), with the
// last W inputs and the W unfinished dx of each channel in registers; dw and dbias are summed
// over the segment's own steps and leave as one partial per segment.
// RAGGED: CPL does not divide the channels.
template <int W, bool BF16, bool DOBF16, bool SILU, int CPL, bool RAGGED>
__global__ __launch_bounds__(64) void conv_bwd_kernel(const char* __restrict__ x, const float* __restrict__ w,
                                                      const float* __restrict__ bias, const char* __restrict__ dout,
                                                      char* __restrict__ dx, float* __restrict__ part,
                                                      CBwdGeo g) {
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
  const int skip = RAGGED ? min(dl - dc, CPL) : 0;  // channels that the lane before has: not stored here
  if (dl >= g.D) return;
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
  const char* const xb = x + (int64_t)b * g.x_batch * ES;
  const char* const db_ = dout + (int64_t)b * g.L * D * DS;
  const int xs = g.dx_bf16 ? 2 : 4;
  const int64_t dxrow = g.dx_row * xs;
  char* const ob = dx + (int64_t)b * g.dx_batch * xs;
  const uint32_t xo = (uint32_t)dc * ES, doff = (uint32_t)dc * DS, oo = (uint32_t)dc * xs;  // the lane's bytes in a row
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = tb - (W - 1) + k;
    RX r;
    if (t >= 0) r.load(xb + (int64_t)t * xrow + xo);
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
      xq[slot][i].template load<true>(row_at(xb, (int64_t)t * xrow), lane_at(xo));
      dq[slot][i].template load<true>(row_at(db_, (int64_t)t * drow), lane_at(doff));
    }
  };
  // Step t; acc[c][k] is the unfinished dx of row t-(W-1)+k.  own: a step of this segment, whose
  // dw and dbias are summed here; else one of the W-1 after it (past: after the sequence's end).
  auto step = [&](const RX& xr, const RD& dr, int t, bool own, bool past) {
    float o[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      win[c][W - 1] = xr.get(c);
      float dv = dr.get(c);
      if constexpr (SILU) {
        float v = bv[c];
#pragma unroll
        for (int k = 0; k < W; ++k) v = __builtin_fmaf(wk[c][k], win[c][k], v);
        const float sg = fast_rcp(1.0f + fast_exp2(-v * kLog2e));
        dv *= sg * __builtin_fmaf(v, 1.0f - sg, 1.0f);
      }
      if (past) dv = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) acc[c][k] = __builtin_fmaf(wk[c][k], dv, acc[c][k]);
      if (own) {
        db[c] += dv;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[c][k] = __builtin_fmaf(dv, win[c][k], dw[c][k]);
      }
      o[c] = acc[c][0];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        acc[c][k] = acc[c][k + 1];
        win[c][k] = win[c][k + 1];
      }
      acc[c][W - 1] = 0.0f;
    }
    const int u = t - (W - 1);
    if (u < tb) return;
    const row_ptr p = row_at(ob, (int64_t)u * dxrow);
    auto put = [&](const auto& r) {  // non-temporal: 4% less time on 2 x 8192 x 5120 than cached
      if constexpr (RAGGED) r.template store_from<true>(p, lane_at(oo), skip);
      else r.template store<true>(p, lane_at(oo));
    };
    if (g.dx_bf16) {
      Vec<true, CPL> r;
      r.set(o);
      put(r);
    } else {
      Vec<false, CPL> r;
      r.set(o);
      put(r);
    }
  };
  load(0, tb);
  int t0 = tb;
  for (; t0 + 2 * kCBwdU <= te; t0 += 2 * kCBwdU) {
    load(1, t0 + kCBwdU);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i) step(xq[0][i], dq[0][i], t0 + i, true, false);
    load(0, t0 + 2 * kCBwdU);
#pragma unroll
    for (int i = 0; i < kCBwdU; ++i) step(xq[1][i], dq[1][i], t0 + kCBwdU + i, true, false);
  }
  // the rest of the segment and the W-1 steps after it
  const int tl = te + W - 1;
  for (; t0 < tl; ++t0) {
    RX xr = xq[0][0];
    RD dr = dq[0][0];
#pragma unroll
    for (int i = 0; i + 1 < kCBwdU; ++i) {
      xq[0][i] = xq[0][i + 1];
      dq[0][i] = dq[0][i + 1];
    }
    const int t = min(t0 + kCBwdU, last);
    xq[0][kCBwdU - 1].load(row_at(xb, (int64_t)t * xrow), lane_at(xo));
    dq[0][kCBwdU - 1].load(row_at(db_, (int64_t)t * drow), lane_at(doff));
    if (t0 < te) step(xr, dr, t0, true, false);
    else step(xr, dr, t0, false, t0 > last);
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
    if constexpr (RAGGED) r.store_from(pp + (int64_t)k * D, skip);
    else r.store(pp + (int64_t)k * D);
  }
}

// dweight (D, W) and dbias (D) from the partials, added in their order
template <int Q>
static __global__ __launch_bounds__(32 * Q) void conv_bwd_sum_kernel(const float* __restrict__ part,
                                                                     float* __restrict__ dw, float* __restrict__ db,
                                                                     int rows, int W, int D) {
  column_sums<Q>(part, rows, (int64_t)(W + 1) * D, [=](int64_t col, float s) {
    const int k = (int)(col / D);
    const int64_t d = col - (int64_t)k * D;
    if (k < W) dw[d * W + k] = s;
    else if (db != nullptr) db[d] = s;
  });
}

ConvBwdPlan plan_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, bool bf16, int num_cus) {
  ConvBwdPlan pl{};
  const int wide = bf16 ? 4 : 2;
  pl.cpl = dim >= wide ? wide : 1;
  const int64_t per_step = batch * ((dim + 64 * pl.cpl - 1) / (64 * pl.cpl));  // waves per time segment
  const int64_t cus = std::max(num_cus, 1);
  // Every segment walks width-1 steps of its neighbours again and leaves a row of partials, so
  // that segments are as long as six waves per CU allow, up to 192 steps (2 x 8192 x 5120 bf16:
  // 110 us with 192 steps, 120 with 64, 122 with 32).  Small layers are bound by one wave's walk and
  // take 32 steps, or 16 or 8 where those would leave most CUs with less than two waves
  // (3 x 1001 x 777 fp32: 16 us with 32 steps, 24 with 64; 64 x 5120: 9.5 with 8, 15 with 32).
  auto waves = [&](int64_t steps) { return per_step * ((seqlen + steps - 1) / steps); };
  const int64_t least = waves(32) >= 2 * cus ? 32 : waves(16) >= 2 * cus ? 16 : 8;
  const int64_t steps = std::max(least, std::min<int64_t>(192, seqlen * per_step / (6 * cus)));
  int64_t S = (seqlen + steps - 1) / steps;
  const int forced = env_int("SSS_FORCE_SEGMENTS", 0);
  if (forced > 0) S = std::min<int64_t>(forced, seqlen);
  pl.seg_len = (seqlen + S - 1) / S;
  pl.segments = (int)((seqlen + pl.seg_len - 1) / pl.seg_len);
  pl.ws_total = (size_t)pl.segments * batch * (width + 1) * dim * 4;
  return pl;
}

template <int W, bool BF16, bool DOBF16, bool SILU, int CPL, bool RAGGED>
static hipError_t run_bwd(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  CBwdGeo g{};
  g.x_row = a.x_row;
  g.x_batch = a.x_batch;
  g.dx_row = a.dx_row;
  g.dx_batch = a.dx_batch;
  g.L = (int)a.seqlen;
  g.D = (int)a.dim;
  g.seg_len = (int)pl.seg_len;
  g.batch = (int)a.batch;
  g.ngroups = (int)((a.dim + 64 * CPL - 1) / (64 * CPL));
  g.dx_bf16 = a.dx_bf16;
  const int64_t grid = (int64_t)g.ngroups * a.batch * pl.segments;
  hipLaunchKernelGGL((conv_bwd_kernel<W, BF16, DOBF16, SILU, CPL, RAGGED>), dim3((unsigned)grid), dim3(64), 0, stream,
                     (const char*)a.x, a.w, a.bias, (const char*)a.dout, (char*)a.dx, (float*)a.workspace, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = (int)(pl.segments * a.batch);
  const dim3 sums(colsum_blocks((int64_t)(W + 1) * a.dim));
  if (colsum_ranges(rows) == 8)
    hipLaunchKernelGGL(conv_bwd_sum_kernel<8>, sums, dim3(256), 0, stream, (const float*)a.workspace, a.dw, a.db, rows, W,
                       (int)a.dim);
  else
    hipLaunchKernelGGL(conv_bwd_sum_kernel<32>, sums, dim3(1024), 0, stream, (const float*)a.workspace, a.dw, a.db, rows,
                       W, (int)a.dim);
  return hipGetLastError();
}

template <int W, bool BF16, bool DOBF16>
static hipError_t run_bwd_shape(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  constexpr int kWide = BF16 ? 4 : 2;  // 8 bytes of x per lane
  if (pl.cpl == 1)
    return a.silu ? run_bwd<W, BF16, DOBF16, true, 1, false>(a, pl, stream)
                  : run_bwd<W, BF16, DOBF16, false, 1, false>(a, pl, stream);
  if (a.dim % kWide == 0)
    return a.silu ? run_bwd<W, BF16, DOBF16, true, kWide, false>(a, pl, stream)
                  : run_bwd<W, BF16, DOBF16, false, kWide, false>(a, pl, stream);
  return a.silu ? run_bwd<W, BF16, DOBF16, true, kWide, true>(a, pl, stream)
                : run_bwd<W, BF16, DOBF16, false, kWide, true>(a, pl, stream);
}

template <int W>
static hipError_t run_bwd_types(const ConvBwdArgs& a, const ConvBwdPlan& pl, hipStream_t stream) {
  if (!a.bf16) return run_bwd_shape<W, false, false>(a, pl, stream);
  return a.dout_bf16 ? run_bwd_shape<W, true, true>(a, pl, stream) : run_bwd_shape<W, true, false>(a, pl, stream);
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

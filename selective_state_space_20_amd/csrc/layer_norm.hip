// layer_norm.hip -- gfx950 kernels of the layer norm over groups of G adjacent channels, forward and gradients,
// alone or after the residual addition (x: the block's output, r: the residual stream):
//   h = x + r  (or x),  hat = (h - mean(h)) rstd(h),  out = hat w + b,  rstd(h) = (mean((h - mean(h))^2) + eps)^-1/2
//   dh = rstd (g - mean(g) - hat mean(g hat)) + dh_out,  g = dout w;  dw = sum dout hat,  db = sum dout
//
// Bound by memory: each element read once and each result written once.  A row (of a group) stays in the registers
// of the lanes that share it, in the shapes of the other norms (norm_rows.h); the variance is summed over the
// deviations from the mean (a second sum over registers), so that a large mean costs no digits.  All sums are fp32.
// bf16 x, fp32 stream, 16384 x 2560: forward 85 us (503 MB, 5.9 TB/s), gradients 120 + 6 us (755 MB, 6.0); bf16 in
// groups of 64, 16384 x 5120, forward 63 us (336 MB, 5.3); 37 x 2560 4 us, one launch and two trips to memory.
#include "norm_rows.h"

#include <algorithm>

namespace sss {

// two sums over the lanes of a row, with one barrier
template <int TPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float* lds, int& turn) {
  if constexpr (TPR <= 64) {
    a = row_sum<TPR>(a, lds, turn);
    b = row_sum<TPR>(b, lds, turn);
  } else {
    a = wave_sum(a);
    b = wave_sum(b);
    constexpr int NW = TPR / 64;
    float* const at = lds + (turn & 1) * 2 * NW;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      at[threadIdx.x >> 6] = a;
      at[NW + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      a += at[i];
      b += at[NW + i];
    }
  }
}

struct LNormGeo {
  int64_t sx, sr;  // elements between rows of x and of the residual
  int64_t rows;
  int64_t step;  // forward: between the rows of a lane
  int G, groups, nblk;
  float eps, inv_g;
};

// residual may be residual_out itself: every element is read by the lane that writes it, before the sums that
// precede the writes.
// R: rows of a lane, `step` apart, so that one load of weight and bias serves all of them.
template <bool XB, bool HB, int V, int TPR, int M, int R>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void layer_norm_fwd_kernel(
    const char* __restrict__ x, const char* residual, const float* __restrict__ w, const float* __restrict__ b,
    char* __restrict__ out, char* residual_out, float* __restrict__ mean_out, float* __restrict__ rstd_out, LNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int XS = XB ? 2 : 4, HS = HB ? 2 : 4;
  static_assert(R == 1 || RPB > 1, "no barrier between the rows of a lane");
  __shared__ float lds[2 * 16];
  // the division in 64 bits once for the workgroup
  const int64_t first = (int64_t)blockIdx.x * RPB, row_first = first / g.groups;
  const unsigned at = (unsigned)(first - row_first * g.groups) + (RPB > 1 ? threadIdx.x / TPR : 0);
  const unsigned down = RPB > 1 ? at / (unsigned)g.groups : 0, grp = at - down * (unsigned)g.groups;
  const int64_t row0 = row_first + down, D = (int64_t)g.G * g.groups;
  if (RPB > 1 && row0 >= g.step) return;  // all lanes of the row; no barrier where a workgroup has many
  const int c0 = (int)grp * g.G;
  const Pieces<V, TPR, M> pc(g.G);
  Vec<XB, V> xr[R][M];
  Vec<HB, V> hr[R][M];
  Vec<false, V> wr[M], br[M];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = R > 1 ? min(row0 + r * g.step, g.rows - 1) : row0;  // past the last: loaded, not used
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      xr[r][m].template load<true>(x + (row * g.sx + c0 + pc.at[m]) * XS);
      if (residual != nullptr) hr[r][m].template load<true>(residual + (row * g.sr + c0 + pc.at[m]) * HS);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
    if (w != nullptr) wr[m].load(w + c0 + pc.at[m]);
    if (b != nullptr) br[m].load(b + c0 + pc.at[m]);
  }
  int turn = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + r * g.step;
    if (R > 1 && row >= g.rows) break;
    float h[M][V], s = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        h[m][c] = xr[r][m].get(c);
        if (residual != nullptr) h[m][c] += hr[r][m].get(c);
        s += c < pc.skip[m] ? 0.0f : h[m][c];
      }
    }
    const float mean = row_sum<TPR>(s, lds, turn) * g.inv_g;
    s = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float d = h[m][c] - mean;
        s += c < pc.skip[m] ? 0.0f : d * d;
      }
    }
    const float rstd = __builtin_amdgcn_rsqf(row_sum<TPR>(s, lds, turn) * g.inv_g + g.eps);
    if ((threadIdx.x & (TPR - 1)) == 0) {
      if (mean_out != nullptr) mean_out[row * g.groups + grp] = mean;
      if (rstd_out != nullptr) rstd_out[row * g.groups + grp] = rstd;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      if (residual_out != nullptr) {
        Vec<HB, V> v;
        v.set(h[m]);
        v.template store_from<false>(residual_out + (row * D + c0 + pc.at[m]) * HS, pc.skip[m]);
      }
      float o[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {  // of h before it is rounded
        o[c] = (h[m][c] - mean) * rstd;
        if (w != nullptr) o[c] *= wr[m].get(c);
        if (b != nullptr) o[c] += br[m].get(c);
      }
      Vec<XB, V> v;
      v.set(o);
      v.template store_from<true>(out + (row * D + c0 + pc.at[m]) * XS, pc.skip[m]);
    }
  }
}

// Gradients.  A workgroup takes every nblk-th set of rows of one group and sums dweight and dbias over them in
// registers; the partials [workgroup][those wanted][D] are added in their order by norm_sum_kernel.
template <bool XB, bool HB, int V, int TPR, int M>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void layer_norm_bwd_kernel(
    const char* __restrict__ dout, const char* __restrict__ dres_out, const char* __restrict__ h,
    const float* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    char* __restrict__ dx, char* __restrict__ dres, float* __restrict__ part, int want_dw, int want_db, LNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int XS = XB ? 2 : 4, HS = HB ? 2 : 4;
  __shared__ float lds[4 * 16];
  const int sub = RPB > 1 ? (int)(threadIdx.x / TPR) : 0;
  const int grp = (int)(blockIdx.x % (unsigned)g.groups);
  const int64_t blk = blockIdx.x / (unsigned)g.groups;
  const int c0 = grp * g.G;
  const int64_t D = (int64_t)g.G * g.groups;
  const Pieces<V, TPR, M> pc(g.G);
  float wv[M][V], dw[M][V], db[M][V];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Vec<false, V> wr;
    wr.zero();
    if (pc.live(m) && w != nullptr) wr.load(w + c0 + pc.at[m]);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      wv[m][c] = w != nullptr ? wr.get(c) : 1.0f;
      dw[m][c] = db[m][c] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t row = blk * RPB + sub; row < g.rows; row += (int64_t)g.nblk * RPB) {
    Vec<XB, V> dr[M];
    Vec<HB, V> hr[M], er[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      dr[m].template load<true>(dout + (row * D + c0 + pc.at[m]) * XS);
      hr[m].template load<true>(h + (row * g.sx + c0 + pc.at[m]) * HS);
      if (dres_out != nullptr) er[m].template load<true>(dres_out + (row * D + c0 + pc.at[m]) * HS);
    }
    const float mean = mean_in[row * g.groups + grp], rstd = rstd_in[row * g.groups + grp];
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float hat = (hr[m].get(c) - mean) * rstd, d = dr[m].get(c), gd = d * wv[m][c];
        dw[m][c] = __builtin_fmaf(d, hat, dw[m][c]);
        db[m][c] += d;
        s += c < pc.skip[m] ? 0.0f : gd;
        q += c < pc.skip[m] ? 0.0f : gd * hat;
      }
    }
    row_sums<TPR>(s, q, lds, turn);
    s *= g.inv_g;
    q *= g.inv_g;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      float dh[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float hat = (hr[m].get(c) - mean) * rstd;
        dh[c] = rstd * (dr[m].get(c) * wv[m][c] - s - hat * q);
        if (dres_out != nullptr) dh[c] += er[m].get(c);
      }
      if (dres != nullptr) {
        Vec<HB, V> r;
        r.set(dh);
        r.template store_from<true>(dres + (row * D + c0 + pc.at[m]) * HS, pc.skip[m]);
      }
      Vec<XB, V> r;
      r.set(dh);
      r.template store_from<true>(dx + (row * D + c0 + pc.at[m]) * XS, pc.skip[m]);
    }
  }
  extern __shared__ float norm_lds[];
  float* pp = part + blk * (want_dw + want_db) * D + c0;
  if (want_dw) put_partials<V, TPR, M>(pp, dw, pc, norm_lds, g.G);
  if (want_db) put_partials<V, TPR, M>(pp + (want_dw ? D : 0), db, pc, norm_lds, g.G);
}

static LNormGeo layer_geo(const LayerNormArgs& a) {
  LNormGeo g{};
  g.sx = a.sx;
  g.sr = a.sr;
  g.rows = a.rows;
  g.G = (int)a.group;
  g.groups = (int)a.groups;
  g.eps = a.eps;
  g.inv_g = 1.0f / (float)a.group;
  return g;
}

// Where a row's lanes are a part of a wave, four rows per lane, from 512 workgroups of them on: weight and bias are twice
// the bytes of a bf16 x each, and came from the caches once per element.  bf16 in groups of 64: 16384 x 5120
// 82 -> 64 us (5.3 TB/s), 1024 x 5120 (640 workgroups) 7.3 -> 6.4, but 256 x 5120 (160) 2.9 -> 3.9; 250 x 40 of 8192
// rows 95 -> 76; groups of 128, 4096 x 16 (1024 workgroups) 9.1 -> 8.6, 1024 x 16 (256) 3.6 -> 4.4.
constexpr int layer_rows(int tpr) { return tpr < 64 ? 4 : 1; }

template <bool XB, bool HB>
static hipError_t layer_fwd(const LayerNormArgs& a, hipStream_t stream) {
  LNormGeo g = layer_geo(a);
  const NormShape sh = norm_shape(a.group, !XB || !HB);
  const int64_t rpb = sh.tpr < 256 ? 256 / sh.tpr : 1;
  const int64_t R = layer_rows(sh.tpr);
  const bool many = R > 1 && a.rows * a.groups >= R * rpb * 512;
  g.step = many ? (a.rows + R - 1) / R : a.rows;
  const dim3 grid((unsigned)((g.step * a.groups + rpb - 1) / rpb));
#define CALL_R(V, TPR, M, R)                                                                                       \
  hipLaunchKernelGGL((layer_norm_fwd_kernel<XB, HB, V, TPR, M, R>), grid, dim3(TPR < 256 ? 256 : TPR), 0, stream,  \
                     (const char*)a.x, (const char*)a.residual, a.w, a.b, (char*)a.out, (char*)a.residual_out, a.mean, \
                     a.rstd, g)
#define CALL(V, TPR, M)                                \
  if (many) CALL_R(V, TPR, M, layer_rows(TPR));        \
  else CALL_R(V, TPR, M, 1)
  SSS_NORM_SHAPES(CALL, !XB || !HB);
#undef CALL
#undef CALL_R
  return hipGetLastError();
}

template <bool XB, bool HB>
static hipError_t layer_bwd(const LayerNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  LNormGeo g = layer_geo(a);
  g.nblk = pl.nblk;
  const NormShape sh = norm_shape(a.group, !XB || !HB);
  const int want_dw = a.dw != nullptr, want_db = a.db != nullptr;
#define CALL(V, TPR, M)                                                                                              \
  hipLaunchKernelGGL((layer_norm_bwd_kernel<XB, HB, V, TPR, M>), dim3((unsigned)(pl.nblk * a.groups)),               \
                     dim3(TPR < 256 ? 256 : TPR), TPR < 256 ? (256 / TPR) * a.group * 4 : 0, stream,                  \
                     (const char*)a.dout, (const char*)a.dres_out, (const char*)a.x, a.w, a.mean, a.rstd, (char*)a.dx, \
                     (char*)a.dres, (float*)a.workspace, want_dw, want_db, g)
  SSS_NORM_SHAPES(CALL, !XB || !HB);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || want_dw + want_db == 0) return e;
  const int64_t D = a.group * a.groups;
  return launch_norm_sum(a.workspace, want_dw ? a.dw : a.db, a.db, nullptr, pl.nblk, D * (want_dw + want_db), D, stream);
}

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, hipStream_t stream) {
  if (a.x_bf16) return a.h_bf16 ? layer_fwd<true, true>(a, stream) : layer_fwd<true, false>(a, stream);
  return a.h_bf16 ? layer_fwd<false, true>(a, stream) : layer_fwd<false, false>(a, stream);
}
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  if (a.x_bf16) return a.h_bf16 ? layer_bwd<true, true>(a, pl, stream) : layer_bwd<true, false>(a, pl, stream);
  return a.h_bf16 ? layer_bwd<false, true>(a, pl, stream) : layer_bwd<false, false>(a, pl, stream);
}

}  // namespace sss

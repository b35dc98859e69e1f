// norms.hip -- gfx950 kernels of the root-mean-square norms around the block, forward and
// gradients.  With rstd(v) = (mean(v^2) + eps)^-1/2 over a group of G adjacent channels:
//
// Gated norm, after the scan (x: the scan's output, z: the block's gate):
//   gate first   u = x silu(z),  out = u rstd(u) w
//   norm first   out = x rstd(x) w silu(z)
// Residual norm, after a block and before the next one (x: the block's output, h: the residual
// stream):
//   v = x rstd(x) wp  (or x),  h' = h + alpha s v,  out = h' rstd(h') w
// Gradients, with hat = u rstd(u) and g the gradient of hat:  du = rstd (g - hat mean(g hat)).
//
// Bound by memory: each element read once and each result written once (16384 x 5120, fp32 x and
// bf16 z: forward 671 MB in 115-121 us, gradients 1174 MB in 233; 16384 x 2560 bf16 with an fp32
// stream: forward 503 MB in 94 us, gradients 755 MB in 134 us).  A row (of a group) is held in
// the registers of 8, 16, 32 or 64 lanes of a wave, or of a workgroup of 256, 512 or 1024 lanes (norm_shape):
// 8 or 4 adjacent elements per lane and piece (16 bytes of bf16 or fp32), M pieces.
// Sums are fp32: lanes of a wave by DPP, waves through LDS.
#include "norm_rows.h"

#include <algorithm>

namespace sss {

struct GNormGeo {
  int64_t sx, sz, sdz;  // elements between rows
  int64_t rows;
  int G, groups, nblk;  // backward: workgroups per group
  float eps, inv_g;
  int norm_first;
};

template <bool XB, bool ZB, int V, int TPR, int M>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void gated_norm_fwd_kernel(
    const char* __restrict__ x, const char* __restrict__ z, const float* __restrict__ w, char* __restrict__ out,
    float* __restrict__ rstd_out, GNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
  constexpr int XS = XB ? 2 : 4, ZS = ZB ? 2 : 4;
  __shared__ float lds[2 * 16];
  const int64_t vr = (int64_t)blockIdx.x * RPB + (RPB > 1 ? (int)(threadIdx.x / TPR) : 0);
  if (RPB > 1 && vr >= g.rows * g.groups) return;  // all lanes of the row; no barrier where a workgroup has many
  const int64_t row = vr / g.groups;
  const int c0 = (int)(vr - row * g.groups) * g.G;
  const Pieces<V, TPR, M> pc(g.G);
  Vec<XB, V> xr[M];
  Vec<ZB, V> zr[M];
  Vec<false, V> wr[M];
  const char* const xp = x + (row * g.sx + c0) * XS;
  const char* const zp = z + (row * g.sz + c0) * ZS;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
    xr[m].template load<true>(xp + (int64_t)pc.at[m] * XS);
    if (z != nullptr) zr[m].template load<true>(zp + (int64_t)pc.at[m] * ZS);
    wr[m].load(w + c0 + pc.at[m]);
  }
  float u[M][V], gt[M][V], s = 0.0f;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      u[m][c] = xr[m].get(c);
      gt[m][c] = z != nullptr ? silu(zr[m].get(c)) : 1.0f;
      if (!g.norm_first) u[m][c] *= gt[m][c];
      s += c < pc.skip[m] ? 0.0f : u[m][c] * u[m][c];
    }
  }
  int turn = 0;
  s = row_sum<TPR>(s, lds, turn);
  const float rstd = __builtin_amdgcn_rsqf(s * g.inv_g + g.eps);
  if (rstd_out != nullptr && (threadIdx.x & (TPR - 1)) == 0) rstd_out[vr] = rstd;
  char* const op = out + (row * (int64_t)g.G * g.groups + c0) * ZS;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
    float o[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      o[c] = u[m][c] * rstd * wr[m].get(c);
      if (g.norm_first) o[c] *= gt[m][c];
    }
    Vec<ZB, V> r;
    r.set(o);
    r.template store_from<true>(op + (int64_t)pc.at[m] * ZS, pc.skip[m]);
  }
}

// Gradients.  A workgroup takes every nblk-th set of rows of one group and sums dweight over them
// in registers; the partials are added in their order by norm_sum_kernel.
template <bool XB, bool ZB, int V, int TPR, int M>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void gated_norm_bwd_kernel(
    const char* __restrict__ dout, const char* __restrict__ x, const char* __restrict__ z, const float* __restrict__ w,
    const float* __restrict__ rstd_in, char* __restrict__ dx, char* __restrict__ dz, float* __restrict__ part,
    GNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int XS = XB ? 2 : 4, ZS = ZB ? 2 : 4;
  __shared__ float lds[2 * 16];
  const int sub = RPB > 1 ? (int)(threadIdx.x / TPR) : 0;
  const int grp = (int)(blockIdx.x % (unsigned)g.groups);
  const int64_t blk = blockIdx.x / (unsigned)g.groups;
  const int c0 = grp * g.G;
  const int64_t D = (int64_t)g.G * g.groups;
  const Pieces<V, TPR, M> pc(g.G);
  float wv[M][V], dw[M][V];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Vec<false, V> wr;
    if (pc.live(m)) wr.load(w + c0 + pc.at[m]);
    else wr.zero();
#pragma unroll
    for (int c = 0; c < V; ++c) {
      wv[m][c] = wr.get(c);
      dw[m][c] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t row = blk * RPB + sub; row < g.rows; row += (int64_t)g.nblk * RPB) {
    Vec<XB, V> xr[M];
    Vec<ZB, V> zr[M], dr[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      dr[m].template load<true>(dout + (row * D + c0 + pc.at[m]) * ZS);
      xr[m].template load<true>(x + (row * g.sx + c0 + pc.at[m]) * XS);
      if (z != nullptr) zr[m].template load<true>(z + (row * g.sz + c0 + pc.at[m]) * ZS);
    }
    const float rstd = rstd_in[row * g.groups + grp];
    float s = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float gate = z != nullptr ? silu(zr[m].get(c)) : 1.0f;
        const float hat = xr[m].get(c) * rstd * (g.norm_first ? 1.0f : gate);
        const float dn = dr[m].get(c) * (g.norm_first ? gate : 1.0f);
        dw[m][c] = __builtin_fmaf(dn, hat, dw[m][c]);
        s += c < pc.skip[m] ? 0.0f : dn * wv[m][c] * hat;
      }
    }
    s = row_sum<TPR>(s, lds, turn) * g.inv_g;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      float ox[V], oz[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float xv = xr[m].get(c), dv = dr[m].get(c);
        float zv = 0.0f, sg = 1.0f, gate = 1.0f;
        if (z != nullptr) {
          zv = zr[m].get(c);
          sg = fast_rcp(1.0f + fast_exp2(-zv * kLog2e));
          gate = zv * sg;
        }
        const float hat = xv * rstd * (g.norm_first ? 1.0f : gate);
        const float gh = dv * (g.norm_first ? gate : 1.0f) * wv[m][c];
        const float du = rstd * (gh - hat * s);
        ox[c] = g.norm_first ? du : du * gate;
        const float dgate = g.norm_first ? dv * hat * wv[m][c] : du * xv;
        oz[c] = dgate * sg * __builtin_fmaf(zv, 1.0f - sg, 1.0f);
      }
      Vec<XB, V> rx;
      rx.set(ox);
      rx.template store_from<true>(dx + (row * D + c0 + pc.at[m]) * XS, pc.skip[m]);
      if (z != nullptr) {
        Vec<ZB, V> rz;
        rz.set(oz);
        rz.template store_from<true>(dz + (row * g.sdz + c0 + pc.at[m]) * ZS, pc.skip[m]);
      }
    }
  }
  extern __shared__ float norm_lds[];
  put_partials<V, TPR, M>(part + blk * D + c0, dw, pc, norm_lds, g.G);
}

struct RNormGeo {
  int64_t sx, sr;  // elements between rows of x and of the residual
  int64_t rows;
  int D, nblk;
  float eps, inv_d, alpha;
};

// The kernel of the residual norm.  POST: x is normed first.  residual may be residual_out itself:
// every element is read by the lane that writes it, before the sum that precedes the writes.
template <bool XB, bool HB, bool POST, int V, int TPR, int M>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void res_norm_fwd_kernel(
    const char* __restrict__ x, const char* residual, const float* __restrict__ wp, const float* __restrict__ scale,
    const float* __restrict__ w, char* __restrict__ out, char* residual_out, float* __restrict__ rstd_post,
    float* __restrict__ rstd_out, RNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int XS = XB ? 2 : 4, HS = HB ? 2 : 4;
  __shared__ float lds[2 * 16];
  const int64_t row = (int64_t)blockIdx.x * RPB + (RPB > 1 ? (int)(threadIdx.x / TPR) : 0);
  if (RPB > 1 && row >= g.rows) return;
  const Pieces<V, TPR, M> pc(g.D);
  Vec<XB, V> xr[M];
  Vec<HB, V> hr[M];
  Vec<false, V> wr[M], pr[M], sr[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
    xr[m].template load<true>(x + (row * g.sx + pc.at[m]) * XS);
    if (residual != nullptr) hr[m].template load<true>(residual + (row * g.sr + pc.at[m]) * HS);
    wr[m].load(w + pc.at[m]);
    if constexpr (POST) pr[m].load(wp + pc.at[m]);
    if (scale != nullptr) sr[m].load(scale + pc.at[m]);
  }
  int turn = 0;
  const bool first = (threadIdx.x & (TPR - 1)) == 0;
  float rp = 1.0f;
  if constexpr (POST) {
    float s = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) s += c < pc.skip[m] ? 0.0f : xr[m].get(c) * xr[m].get(c);
    }
    s = row_sum<TPR>(s, lds, turn);
    rp = __builtin_amdgcn_rsqf(s * g.inv_d + g.eps);
    if (rstd_post != nullptr && first) rstd_post[row] = rp;
  }
  float h[M][V], s = 0.0f;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float v = xr[m].get(c);
      if constexpr (POST) v *= rp * pr[m].get(c);
      v *= scale != nullptr ? g.alpha * sr[m].get(c) : g.alpha;
      h[m][c] = residual != nullptr ? hr[m].get(c) + v : v;
      s += c < pc.skip[m] ? 0.0f : h[m][c] * h[m][c];
    }
  }
  s = row_sum<TPR>(s, lds, turn);
  const float rstd = __builtin_amdgcn_rsqf(s * g.inv_d + g.eps);
  if (rstd_out != nullptr && first) rstd_out[row] = rstd;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!pc.live(m)) continue;
    Vec<HB, V> rh;
    rh.set(h[m]);
    rh.template store_from<false>(residual_out + (row * (int64_t)g.D + pc.at[m]) * HS, pc.skip[m]);
    float o[V];
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = h[m][c] * rstd * wr[m].get(c);  // of h' before it is rounded
    Vec<XB, V> r;
    r.set(o);
    r.template store_from<true>(out + (row * (int64_t)g.D + pc.at[m]) * XS, pc.skip[m]);
  }
}

// Gradients; partials [workgroup][up to 3][D]: dweight, dpost_weight, dscale (those that are wanted).
template <bool XB, bool HB, bool POST, int V, int TPR, int M>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void res_norm_bwd_kernel(
    const char* __restrict__ dout, const char* __restrict__ dres_out, const char* __restrict__ x,
    const char* __restrict__ h, const float* __restrict__ wp, const float* __restrict__ scale,
    const float* __restrict__ w, const float* __restrict__ rstd_post, const float* __restrict__ rstd_in,
    char* __restrict__ dx, char* __restrict__ dres, float* __restrict__ part, RNormGeo g) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int XS = XB ? 2 : 4, HS = HB ? 2 : 4;
  __shared__ float lds[2 * 16];
  const int sub = RPB > 1 ? (int)(threadIdx.x / TPR) : 0;
  const int64_t blk = blockIdx.x;
  const int64_t D = g.D;
  const Pieces<V, TPR, M> pc(g.D);
  const bool use_x = POST || scale != nullptr;
  float wv[M][V], pv[M][V], sv[M][V], dw[M][V], dp[M][V], ds[M][V];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Vec<false, V> a, b, c2;
    a.zero();
    b.zero();
    c2.zero();
    if (pc.live(m)) {
      a.load(w + pc.at[m]);
      if constexpr (POST) b.load(wp + pc.at[m]);
      if (scale != nullptr) c2.load(scale + pc.at[m]);
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      wv[m][c] = a.get(c);
      pv[m][c] = POST ? b.get(c) : 1.0f;
      sv[m][c] = scale != nullptr ? g.alpha * c2.get(c) : g.alpha;
      dw[m][c] = dp[m][c] = ds[m][c] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t row = blk * RPB + sub; row < g.rows; row += (int64_t)g.nblk * RPB) {
    Vec<XB, V> dr[M], xr[M];
    Vec<HB, V> hr[M], er[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      dr[m].template load<true>(dout + (row * D + pc.at[m]) * XS);
      hr[m].template load<true>(h + (row * D + pc.at[m]) * HS);
      if (dres_out != nullptr) er[m].template load<true>(dres_out + (row * D + pc.at[m]) * HS);
      if (use_x) xr[m].template load<true>(x + (row * g.sx + pc.at[m]) * XS);
    }
    const float rstd = rstd_in[row];
    float s = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float hat = hr[m].get(c) * rstd, d = dr[m].get(c);
        dw[m][c] = __builtin_fmaf(d, hat, dw[m][c]);
        s += c < pc.skip[m] ? 0.0f : d * wv[m][c] * hat;
      }
    }
    s = row_sum<TPR>(s, lds, turn) * g.inv_d;
    float dh[M][V];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float hat = hr[m].get(c) * rstd;
        const float d = rstd * (dr[m].get(c) * wv[m][c] - hat * s);
        dh[m][c] = dres_out != nullptr ? er[m].get(c) + d : d;
      }
      if (dres != nullptr) {
        Vec<HB, V> r;
        r.set(dh[m]);
        r.template store_from<true>(dres + (row * D + pc.at[m]) * HS, pc.skip[m]);
      }
    }
    const float rp = POST ? rstd_post[row] : 1.0f;
    float s2 = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float hat = use_x ? xr[m].get(c) * rp : 0.0f;  // x rstd(x), or x
        const float dv = sv[m][c] * dh[m][c];
        if (scale != nullptr) ds[m][c] = __builtin_fmaf(g.alpha * dh[m][c], hat * pv[m][c], ds[m][c]);
        if constexpr (POST) {
          dp[m][c] = __builtin_fmaf(dv, hat, dp[m][c]);
          s2 += c < pc.skip[m] ? 0.0f : dv * pv[m][c] * hat;
        }
      }
    }
    if constexpr (POST) s2 = row_sum<TPR>(s2, lds, turn) * g.inv_d;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      float o[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float dv = sv[m][c] * dh[m][c];
        if constexpr (POST) o[c] = rp * (dv * pv[m][c] - xr[m].get(c) * rp * s2);
        else o[c] = dv;
      }
      Vec<XB, V> r;
      r.set(o);
      r.template store_from<true>(dx + (row * D + pc.at[m]) * XS, pc.skip[m]);
    }
  }
  const int64_t vecs = 1 + (POST ? 1 : 0) + (scale != nullptr ? 1 : 0);
  extern __shared__ float norm_lds[];
  float* pp = part + blk * vecs * D;
  put_partials<V, TPR, M>(pp, dw, pc, norm_lds, g.D);
  if constexpr (POST) put_partials<V, TPR, M>(pp += D, dp, pc, norm_lds, g.D);
  if (scale != nullptr) put_partials<V, TPR, M>(pp += D, ds, pc, norm_lds, g.D);
}

int norm_lanes(int64_t group, bool fp32) { return norm_shape(group, fp32).tpr; }

NormPlan plan_norm_bwd(int64_t rows, int64_t group, int64_t groups, int vectors, bool fp32, int num_cus) {
  NormPlan pl{};
  const NormShape sh = norm_shape(group, fp32);
  const int rpb = sh.tpr < 256 ? 256 / sh.tpr : 1;
  // Four workgroups per CU (two of more than 256 lanes), but six rows for each as long as every CU
  // has one: a workgroup leaves a row of partials for each vector of parameters (3000 x 5121
  // fp32 with three of them: 108 us with six rows, 121 with three).  No more than there are sets of
  // the rows that a workgroup takes at once, 32 of the shortest groups'.
  const int64_t sets = std::max<int64_t>(1, (rows + rpb - 1) / rpb), cus = std::max(num_cus, 1);
  const int64_t want = std::max<int64_t>(1, cus * (sh.tpr > 256 ? 2 : 4) / groups);
  const int64_t one_each = std::max<int64_t>(1, std::min<int64_t>(sets, cus / groups));
  pl.nblk = (int)std::min({want, sets, std::max<int64_t>(one_each, rows / 6)});
  pl.ws_total = (size_t)pl.nblk * vectors * group * groups * 4;
  return pl;
}

static GNormGeo gated_geo(const GatedNormArgs& a) {
  GNormGeo g{};
  g.sx = a.sx;
  g.sz = a.sz;
  g.sdz = a.sdz;
  g.rows = a.rows;
  g.G = (int)a.group;
  g.groups = (int)a.groups;
  g.eps = a.eps;
  g.inv_g = 1.0f / (float)a.group;
  g.norm_first = a.norm_first;
  return g;
}

template <bool XB, bool ZB>
static hipError_t gated_fwd(const GatedNormArgs& a, hipStream_t stream) {
  const GNormGeo g = gated_geo(a);
  const NormShape sh = norm_shape(a.group, !XB || !ZB);
  const int64_t vrows = a.rows * a.groups;
#define CALL(V, TPR, M)                                                                                             \
  hipLaunchKernelGGL((gated_norm_fwd_kernel<XB, ZB, V, TPR, M>),                                                    \
                     dim3((unsigned)((vrows + (TPR < 256 ? 256 / TPR : 1) - 1) / (TPR < 256 ? 256 / TPR : 1))),      \
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, (const char*)a.x, (const char*)a.z, a.w, (char*)a.out, \
                     a.rstd, g)
  SSS_NORM_SHAPES(CALL, !XB || !ZB);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t stream) {
  if (a.x_bf16) return a.z_bf16 ? gated_fwd<true, true>(a, stream) : gated_fwd<true, false>(a, stream);
  return a.z_bf16 ? gated_fwd<false, true>(a, stream) : gated_fwd<false, false>(a, stream);
}

template <bool XB, bool ZB>
static hipError_t gated_bwd(const GatedNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  GNormGeo g = gated_geo(a);
  g.nblk = pl.nblk;
  const NormShape sh = norm_shape(a.group, !XB || !ZB);
#define CALL(V, TPR, M)                                                                                               \
  hipLaunchKernelGGL((gated_norm_bwd_kernel<XB, ZB, V, TPR, M>), dim3((unsigned)(pl.nblk * a.groups)),                 \
                     dim3(TPR < 256 ? 256 : TPR), TPR < 256 ? (256 / TPR) * a.group * 4 : 0, stream, (const char*)a.dout, (const char*)a.x, (const char*)a.z, \
                     a.w, a.rstd, (char*)a.dx, (char*)a.dz, (float*)a.workspace, g)
  SSS_NORM_SHAPES(CALL, !XB || !ZB);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t D = a.group * a.groups;
  return launch_norm_sum(a.workspace, a.dw, nullptr, nullptr, pl.nblk, D, D, stream);
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  if (a.x_bf16) return a.z_bf16 ? gated_bwd<true, true>(a, pl, stream) : gated_bwd<true, false>(a, pl, stream);
  return a.z_bf16 ? gated_bwd<false, true>(a, pl, stream) : gated_bwd<false, false>(a, pl, stream);
}

static RNormGeo res_geo(const ResNormArgs& a) {
  RNormGeo g{};
  g.sx = a.sx;
  g.sr = a.sr;
  g.rows = a.rows;
  g.D = (int)a.dim;
  g.eps = a.eps;
  g.inv_d = 1.0f / (float)a.dim;
  g.alpha = a.alpha;
  return g;
}

template <bool XB, bool HB, bool POST>
static hipError_t res_fwd(const ResNormArgs& a, hipStream_t stream) {
  const RNormGeo g = res_geo(a);
  const NormShape sh = norm_shape(a.dim, !XB || !HB);
#define CALL(V, TPR, M)                                                                                               \
  hipLaunchKernelGGL((res_norm_fwd_kernel<XB, HB, POST, V, TPR, M>),                                                  \
                     dim3((unsigned)((a.rows + (TPR < 256 ? 256 / TPR : 1) - 1) / (TPR < 256 ? 256 / TPR : 1))),       \
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, (const char*)a.x, (const char*)a.residual, a.wp, a.scale, \
                     a.w, (char*)a.out, (char*)a.residual_out, a.rstd_post, a.rstd, g)
  SSS_NORM_SHAPES(CALL, !XB || !HB);
#undef CALL
  return hipGetLastError();
}

template <bool XB, bool HB, bool POST>
static hipError_t res_bwd(const ResNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  RNormGeo g = res_geo(a);
  g.nblk = pl.nblk;
  const NormShape sh = norm_shape(a.dim, !XB || !HB);
#define CALL(V, TPR, M)                                                                                                \
  hipLaunchKernelGGL((res_norm_bwd_kernel<XB, HB, POST, V, TPR, M>), dim3((unsigned)pl.nblk),                          \
                     dim3(TPR < 256 ? 256 : TPR), TPR < 256 ? (256 / TPR) * a.dim * 4 : 0, stream, (const char*)a.dout, (const char*)a.dres_out,             \
                     (const char*)a.x, (const char*)a.residual_out, a.wp, a.scale, a.w, a.rstd_post, a.rstd,           \
                     (char*)a.dx, (char*)a.dres, (float*)a.workspace, g)
  SSS_NORM_SHAPES(CALL, !XB || !HB);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t cols = a.dim * (1 + (POST ? 1 : 0) + (a.scale != nullptr ? 1 : 0));
  return launch_norm_sum(a.workspace, a.dw, POST ? a.dwp : a.dscale, a.dscale, pl.nblk, cols, a.dim, stream);
}

template <bool XB, bool HB>
static hipError_t res_types(const ResNormArgs& a, const NormPlan* pl, hipStream_t stream) {
  if (a.wp != nullptr) return pl ? res_bwd<XB, HB, true>(a, *pl, stream) : res_fwd<XB, HB, true>(a, stream);
  return pl ? res_bwd<XB, HB, false>(a, *pl, stream) : res_fwd<XB, HB, false>(a, stream);
}

static hipError_t res_norm(const ResNormArgs& a, const NormPlan* pl, hipStream_t stream) {
  if (a.x_bf16) return a.h_bf16 ? res_types<true, true>(a, pl, stream) : res_types<true, false>(a, pl, stream);
  return a.h_bf16 ? res_types<false, true>(a, pl, stream) : res_types<false, false>(a, pl, stream);
}

hipError_t launch_res_norm_fwd(const ResNormArgs& a, hipStream_t stream) { return res_norm(a, nullptr, stream); }
hipError_t launch_res_norm_bwd(const ResNormArgs& a, const NormPlan& pl, hipStream_t stream) {
  return res_norm(a, &pl, stream);
}

}  // namespace sss

// norm_rows.h -- rows of a norm in registers: sums over the lanes that share a row, its pieces, partial parameter
// gradients and their sums, and the shapes of the kernels (norms.hip, layer_norm.hip).
#pragma once
#include "colsum.h"
#include "vec.h"
#include "kernels.h"

namespace sss {

template <int CTRL>
__device__ __forceinline__ float norm_dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float norm_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
// sum over a wave, the same in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += norm_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v += norm_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v += norm_dpp<0x141>(v);  // row_half_mirror
  v += norm_dpp<0x140>(v);  // row_mirror: each row of 16 lanes holds its sum
  return (norm_lane(v, 0) + norm_lane(v, 16)) + (norm_lane(v, 32) + norm_lane(v, 48));
}

// Sum over the TPR lanes that share a row.  `turn` alternates the LDS buffer: a wave that
// writes a buffer again has passed the barrier of the sum in between, before which every
// wave has read it, so that one barrier per sum suffices.
// Up to 64 lanes per row are a wave or an aligned part of one.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* lds, int& turn) {
  if constexpr (TPR < 64) {
    v += norm_dpp<0xB1>(v);
    v += norm_dpp<0x4E>(v);
    v += norm_dpp<0x141>(v);
    if constexpr (TPR >= 16) v += norm_dpp<0x140>(v);
    if constexpr (TPR >= 32) v += __shfl_xor(v, 16);
    return v;
  }
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    float* const b = lds + (turn & 1) * NW;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += b[i];
  }
  return v;
}

// The pieces of a row of G elements: piece p starts at element V p, the last one V elements
// before the row's end where V does not divide G: its first `skip` elements are then another
// lane's, count for nothing and are not stored.
template <int V, int TPR, int M>
struct Pieces {
  int at[M], skip[M];
  __device__ __forceinline__ Pieces(int G) {
    const int tid = (int)threadIdx.x & (TPR - 1);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int p = (m * TPR + tid) * V;
      at[m] = min(p, G - V);
      skip[m] = min(p - at[m], V);
    }
  }
  __device__ __forceinline__ bool live(int m) const { return skip[m] < V; }
};

// One row of partial parameter gradients per workgroup: where each wave has rows of its own, the
// waves' sums are joined in LDS first, in their order (RPB * G floats of it).
template <int V, int TPR, int M>
__device__ __forceinline__ void put_partials(float* __restrict__ to, const float (&v)[M][V], const Pieces<V, TPR, M>& pc,
                                             float* lds, int G) {
  if constexpr (TPR >= 256) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (!pc.live(m)) continue;
      Vec<false, V> r;
      r.set(v[m]);
      r.store_from(to + pc.at[m], pc.skip[m]);
    }
  } else {
    constexpr int RPB = 256 / TPR;
    float* const mine = lds + (threadIdx.x / TPR) * G;
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int c = 0; c < V; ++c)
        if (pc.live(m) && c >= pc.skip[m]) mine[pc.at[m] + c] = v[m][c];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G; i += 256) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < RPB; ++q) s += lds[q * G + i];
      to[i] = s;
    }
    __syncthreads();
  }
}

// Parameter gradients from the partials, added in their order: columns d, D + d, 2D + d are those
// of out0, out1, out2.
template <int Q>
static __global__ __launch_bounds__(32 * Q) void norm_sum_kernel(const float* __restrict__ part, float* __restrict__ out0,
                                                                 float* __restrict__ out1, float* __restrict__ out2,
                                                                 int rows, int64_t cols, int D) {
  column_sums<Q>(part, rows, cols, [=](int64_t col, float s) {
    if (col < D) out0[col] = s;
    else if (col < 2 * (int64_t)D) out1[col - D] = s;
    else out2[col - 2 * (int64_t)D] = s;
  });
}

static hipError_t launch_norm_sum(const void* part, float* out0, float* out1, float* out2, int rows, int64_t cols,
                                  int64_t D, hipStream_t stream) {
  const dim3 grid(colsum_blocks(cols));
  if (colsum_ranges(rows) == 8)
    hipLaunchKernelGGL(norm_sum_kernel<8>, grid, dim3(256), 0, stream, (const float*)part, out0, out1, out2, rows, cols,
                       (int)D);
  else
    hipLaunchKernelGGL(norm_sum_kernel<32>, grid, dim3(1024), 0, stream, (const float*)part, out0, out1, out2, rows, cols,
                       (int)D);
  return hipGetLastError();
}

// Lanes per row and pieces per lane for rows of G elements, V elements per piece.  V = 8 is 16 bytes
// of bf16.  Where a tensor is fp32, V = 4 makes every access of it 16 adjacent bytes per lane instead of
// two accesses of every other 16: forward of 16384 x 5120, fp32 x and bf16 z, 129 -> 114 us;
// residual norm of 16384 x 2560 with an fp32 stream, forward 110 -> 94 us, gradients 144 -> 136.
// At most three pieces per lane, then 512 lanes: with five of V = 4 the gradients' registers leave few
// waves (gated forward and gradients of 16384 x 5120 332 us on 512 lanes, 402 on 256, 372 with V =
// 8 on 256; x 2560 174 on 256 lanes with three pieces, 187 on 512 with two; residual norm x 4096 383 on
// 512, 421 on 256 with four).  Above 6144 elements V = 4 would need 1024 lanes.  Pieces of V = 8 follow
// the same rule on the evidence of one forward alone (bf16 x 8192: 185 us on 512 lanes, 188 on 256
// with four): their residual gradients at 4097 to 6144 elements need 272 to 320 registers, one wave per
// SIMD (16384 x 5120, bf16 stream: 263 us, 3.8 TB/s), and have not been measured on 512 lanes.  Fewer than 8 elements: one each, 8 lanes.
//
// Shapes that do not fit their registers: the residual gradients from 8193 elements on (15 to 145
// registers of a lane in scratch memory up to 12288, 106 to 497 up to 16384, 391 to 816 above); all
// other kernels above 16384 (gated forward 16, residual forward 8 to 157, gated gradients 158 to 252),
// and the gated gradients of two fp32 tensors from 12289 on (4).
struct NormShape {
  int v, tpr, m;
};
static NormShape norm_shape(int64_t G, bool fp32) {
  if (G < 8) return {1, 8, 1};
  const int v = fp32 && G <= 6144 ? 4 : 8;
  const int64_t p = (G + v - 1) / v;
  if (p <= 8) return {v, 8, 1};  // 16384 x 5120 in groups of 64: forward 421 us with a wave per row
  if (p <= 16) return {v, 16, 1};
  if (p <= 32) return {v, 32, 1};
  if (p <= 64) return {v, 64, 1};
  if (p <= 128) return {v, 64, 2};
  if (p <= 768) return {v, 256, (int)((p + 255) / 256)};
  if (p <= 2048) return {v, 512, (int)((p + 511) / 512)};
  return {v, 1024, 4};
}

// CALL(V, TPR, M) of the shape sh, of those that norm_shape gives; F32: one of the tensors is fp32.
// Each chain ends in an else: no shape is without a kernel.
#define SSS_NORM_UP_TO_256(CALL, V)                                             \
  if (sh.tpr == 8) { CALL(V, 8, 1); }                                           \
  else if (sh.tpr == 16) { CALL(V, 16, 1); }                                    \
  else if (sh.tpr == 32) { CALL(V, 32, 1); }                                    \
  else if (sh.tpr == 64 && sh.m == 1) { CALL(V, 64, 1); }                       \
  else if (sh.tpr == 64) { CALL(V, 64, 2); }                                    \
  else if (sh.tpr == 256 && sh.m == 1) { CALL(V, 256, 1); }                     \
  else if (sh.tpr == 256 && sh.m == 2) { CALL(V, 256, 2); }                     \
  else if (sh.tpr == 256) { CALL(V, 256, 3); }
#define SSS_NORM_SHAPES(CALL, F32)                                              \
  do {                                                                          \
    if (sh.v == 1) {                                                            \
      CALL(1, 8, 1);                                                            \
    } else if (sh.v == 4) { /* up to 1536 pieces, with an fp32 tensor only */   \
      if constexpr (F32) {                                                      \
        SSS_NORM_UP_TO_256(CALL, 4)                                             \
        else if (sh.m == 2) { CALL(4, 512, 2); }                                \
        else { CALL(4, 512, 3); }                                               \
      }                                                                         \
    } else {                                                                    \
      if constexpr (!F32) { /* with one from 769 pieces on only */              \
        SSS_NORM_UP_TO_256(CALL, 8)                                             \
        if (sh.tpr <= 256) break;                                               \
      }                                                                         \
      if (sh.tpr == 512 && sh.m == 2) { CALL(8, 512, 2); }                      \
      else if (sh.tpr == 512 && sh.m == 3) { CALL(8, 512, 3); }                 \
      else if (sh.tpr == 512) { CALL(8, 512, 4); }                              \
      else { CALL(8, 1024, 4); }                                                \
    }                                                                           \
  } while (0)

}  // namespace sss

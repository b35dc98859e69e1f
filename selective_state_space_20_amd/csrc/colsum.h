// colsum.h -- column sums of partial results, in a fixed order (HIP, gfx950).
//
// The gradients of parameters are summed over rows by many workgroups, each leaving one row of
// partials; here `rows` such rows of `cols` floats are added.  A workgroup takes 32 adjacent
// columns (128-byte pieces of a row) and splits the rows in Q ranges, one per 32 lanes, 16 loads
// in flight each; the ranges are joined in LDS in their order.
#pragma once
#include "common.h"

namespace sss {

// Q = 8 (256 lanes) up to 128 rows, else 32 (1024 lanes).
inline int colsum_ranges(int rows) { return rows <= 128 ? 8 : 32; }
inline unsigned colsum_blocks(int64_t cols) { return (unsigned)((cols + 31) / 32); }

// out(col, sum) for every column of this workgroup, by its first 32 lanes
template <int Q, typename Out>
__device__ __forceinline__ void column_sums(const float* __restrict__ part, int rows, int64_t cols, Out out) {
  __shared__ float lds[Q * 32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int64_t cc = min(col, cols - 1);
  const int per = (rows + Q - 1) / Q;
  const int r0 = q * per, r1 = min(rows, r0 + per);
  constexpr int B = 16;
  float s = 0.0f;
  for (int r = r0; r < r1; r += B) {
    float v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = part[(int64_t)min(r + i, r1 - 1) * cols + cc];
#pragma unroll
    for (int i = 0; i < B; ++i) s += r + i < r1 ? v[i] : 0.0f;
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (q != 0 || col >= cols) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < Q; ++i) t += lds[i * 32 + lane];
  out(col, t);
}

}  // namespace sss

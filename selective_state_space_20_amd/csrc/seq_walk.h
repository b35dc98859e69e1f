// seq_walk.h -- which rows of a packed batch a chunk works on (host and device: plain integers,
// so that the CPU tests run the same lines over any boundaries).
//
// Boundaries come from the caller's device memory and are never trusted for an address: a
// batch is cut at what lies in [0, tokens], and a sequence that a chunk meets at row t began
// either in an earlier chunk or at t.
#pragma once

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define SSS_HD __host__ __device__ __forceinline__
#else
#define SSS_HD inline
#endif

namespace sss {

// The sequence with first boundary cu_s began before the chunk at row c0: an earlier chunk has
// worked on it.  Never so in the first chunk.
SSS_HD bool began_before(int cu_s, int c0) { return (cu_s > 0 ? cu_s : 0) < c0; }

// What a chunk [.., tend) of the convolution does at its row t, which lies in the sequence with
// first boundary cu_s and last row `end` - 1 (end > t); H rows of history per tap line.
struct ConvPiece {
  int beg;    // the sequence's first row, t or before the chunk
  int next;   // the row to go on at
  bool mine;  // rows t .. next - 1 are computed here; else an earlier chunk has them
};

// The first H rows of a sequence belong to the chunk that holds its start, also where they pass
// that chunk's end (tend).  A piece that is `mine` therefore starts at t == beg, with its history
// in the cache, or at t >= beg + H, with the H rows before t in the sequence: t - H >= beg >= 0.
SSS_HD ConvPiece conv_piece(int cu_s, int end, int t, int c0, int tend, int H) {
  if (!began_before(cu_s, c0)) {  // it begins at t, whatever its boundary says
    const int reach = t + H > tend ? t + H : tend;
    return {t, end < reach ? end : reach, true};
  }
  const int beg = cu_s > 0 ? cu_s : 0;
  if (t - beg < H) return {beg, end < beg + H ? end : beg + H, false};
  return {beg, end < tend ? end : tend, true};
}

}  // namespace sss

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

}  // namespace sss

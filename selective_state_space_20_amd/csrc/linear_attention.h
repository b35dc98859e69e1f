// linear_attention.h -- what the host and the kernels of linear attention with a decay for each
// head share (linear_attention.hip: the walks on the matrix cores; linear_attention_parts.hip: what
// stands between and after them, and the single-token step).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "vec.h"

namespace sss {

constexpr int kLaTile = 64;  // tokens of a tile (bf16); fp32 takes 32
constexpr float kLaCut = -1e4f;  // a log decay up to this leaves nothing of the state, whatever those beside it

// One operand of (tokens, heads, width): elements between tokens and between heads, and how many
// of the call's heads share one of its heads.
struct LaSide {
  const char* p;
  int64_t st, sh;
  int rep, width;
};

// A walk over the tokens of a segment, for one head (see linear_attention.hip).
struct LaWalk {
  LaSide x, y, z, w;
  char* out;
  int64_t out_st, out_sh;
  int out_f32;  // partial results of shared heads, kept in fp32
  const float* g;
  int64_t g_st;  // 0: one decay per head
  const float* beta;  // nullable
  int64_t beta_st;
  const float* D;  // nullable
  float scale;
  const int32_t* cu;
  const int32_t* sidx;  // nullable
  const uint8_t* init;  // nullable
  float* state;         // slots: read at a sequence's start, written at its end; nullable
  const float* from;    // gradients: per sequence, the state (adjoint) to start from; nullable
  float* to;            // gradients: per sequence, where the adjoint at its start goes; nullable
  int64_t se, sf;       // elements of a state between rows e and columns f
  int64_t hs;           // elements of a head's state
  float* end;           // [segment][head][hs] of the sequence that runs across the segment's edge
  float* begin;         // [segment][head][hs] of its first state where it begins in the segment
  const float* enter;   // [segment][head][hs] entering the segment
  const float* back;    // [segment][head][hs] adjoint entering the segment from the right
  const float* dfinal;  // per sequence, nullable
  float* sum;           // [segment][head] log2 of the decay over the folded part
  int32_t* flag;        // [segment]
  // [head][tokens], of the pairs of tokens whose products make dg and db:
  float* rows;          // q . dq from earlier tiles
  float* cols;          // k . dk / beta within the tile
  float* cols2;         // the same from later tiles
  float* within;        // dg of the pairs within the tile
  // <adjoint behind, state before> the last tile of a segment's part of a sequence, decayed over the tile: the part
  // of its tokens' dg from tokens on both sides of it
  float* edge;          // [segment][head] of the sequence that runs across the segment's right edge
  float* last;          // [sequence][head] of those that end
  float* trace;         // [segment][head] sum of dout . v
  int tokens, nseq, slots, H, K, nseg;
};

enum LaMode { kLaFoldFwd, kLaFoldRev, kLaFwd, kLaDq, kLaDk, kLaDv };

// E: rows of the walk's state (the width of x and y), F: its columns (that of z and out), rounded
// up to 64, 128 or 256.
hipError_t la_launch(int E, int F, LaMode mode, bool bf16, const LaWalk& g, unsigned grid, hipStream_t stream);
// Both folds (kLaFoldFwd, kLaFoldRev), n workgroups each; and dq and dk, and where E is F also dv.
hipError_t la_launch_folds(int E, int F, bool bf16, const LaWalk& fwd, const LaWalk& rev, unsigned n, hipStream_t stream);
hipError_t la_launch_grads(int E, int F, bool bf16, const LaWalk& dq, const LaWalk& dk, const LaWalk& dv, unsigned n,
                           hipStream_t stream);

// States between segments: enter[c + 1] from end, sum and flag of segment c; of a second set, if any, enter[c - 1].
struct LaCarry {
  const float* end;
  const float* sum;
  const int32_t* flag;
  float* enter;
};
hipError_t la_carry(const LaCarry& fwd, const LaCarry* rev, int64_t hs, int H, int nseg, hipStream_t stream);

// dlog_decay and dbeta from what the walks leave, and dD: see linear_attention_parts.hip
struct LaFinish {
  const float* rows;  // see LaWalk
  const float* cols;
  const float* cols2;
  const float* within;
  const float* edge;
  const float* last;
  const float* g;
  int64_t g_st;
  const float* beta;
  int64_t beta_st;
  const int32_t* cu;
  float* dg;     // (tokens, heads), or with part: (heads)
  float* part;   // [segment][head]: one decay per head; else null
  float* dbeta;  // nullable
  const float* trace;
  float* dD;  // nullable
  int tokens, nseq, H, K, nseg, tile;
};
hipError_t la_finish(const LaFinish& a, hipStream_t stream);

// out (tokens, heads / rep, d) = sums of rep adjacent heads of part (tokens, heads, d); of a second set, if any, too
struct LaSum {
  const float* part;
  void* out;
  int rep;
};
hipError_t la_sum_heads(const LaSum& a, const LaSum* b, int64_t tokens, int heads, int d, bool bf16, hipStream_t stream);
// dinitial = dfinal (or zero) of the sequences without tokens
hipError_t la_empty(const int32_t* cu, const float* dfinal, float* dinitial, int nseq, int tokens, int64_t per, hipStream_t stream);

struct LaStep {
  LaSide q, k, v;
  char* out;
  const float* g;
  int64_t g_st;
  const float* beta;
  int64_t beta_st;
  const float* D;
  float scale;
  float* state;
  const int32_t* sidx;
  int64_t rows;
  int slots, H;
};
hipError_t la_step(const LaStep& a, bool bf16, hipStream_t stream);

template <int E, int F>
hipError_t la_run_folds(bool bf16, const LaWalk& fwd, const LaWalk& rev, unsigned n, hipStream_t stream);
template <int E, int F>
hipError_t la_run_grads(bool bf16, const LaWalk& dq, const LaWalk& dk, const LaWalk& dv, unsigned n, hipStream_t stream);
template <int E, int F>
hipError_t la_run(LaMode mode, bool bf16, const LaWalk& g, unsigned grid, hipStream_t stream);

#ifdef __HIPCC__
// The boundaries of a packed batch, in a wave's lanes where there are at most 64, so that a walk over its sequences
// waits for memory once.  All lanes take part in each call; s and t are the same in all.
struct LaBounds {
  const int32_t* cu;
  int nseq, lane, mine;
  __device__ __forceinline__ LaBounds(const int32_t* cu_, int nseq_, int lane_) : cu(cu_), nseq(nseq_), lane(lane_) {
    mine = cu[min(lane, nseq)];
  }
  __device__ __forceinline__ int at(int s) const {
    return nseq < 64 ? __builtin_amdgcn_readlane(mine, s) : __builtin_amdgcn_readfirstlane(cu[s]);
  }
  // the last sequence that begins at t or before
  __device__ __forceinline__ int find(int t) const {
    const int s = nseq < 64 ? __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane <= nseq && mine <= t)) - 1
                            : __builtin_amdgcn_readfirstlane(find_seq(cu, nseq, t, lane));
    return min(max(s, 0), nseq - 1);
  }
};

#endif

}  // namespace sss

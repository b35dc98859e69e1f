// linear_attention_parts.hip -- gfx950 kernels around the walks of linear_attention.hip: the states that
// enter segments, the gradients of the decays, sums over shared heads, and the single-token step.
#include "linear_attention.h"

#include "colsum.h"
#include "vec.h"

#include <algorithm>

namespace sss {

// Walks are compiled once per pair of sizes (build.py).
#define SSS_LA_EXTERN(E, F)                                                                                          \
  extern template hipError_t la_run<E, F>(LaMode, bool, const LaWalk&, unsigned, hipStream_t);                       \
  extern template hipError_t la_run_folds<E, F>(bool, const LaWalk&, const LaWalk&, unsigned, hipStream_t);          \
  extern template hipError_t la_run_grads<E, F>(bool, const LaWalk&, const LaWalk&, const LaWalk&, unsigned, hipStream_t);
#define SSS_LA_SIZES(CALL) \
  CALL(64, 64) CALL(64, 128) CALL(64, 256) CALL(128, 64) CALL(128, 128) CALL(128, 256) CALL(256, 64) CALL(256, 128) CALL(256, 256)
SSS_LA_SIZES(SSS_LA_EXTERN)
#undef SSS_LA_EXTERN

#define SSS_LA_PICK(NAME, ...)                                      \
  do {                                                              \
    if (E == 64 && F == 64) return NAME<64, 64>(__VA_ARGS__);       \
    if (E == 64 && F == 128) return NAME<64, 128>(__VA_ARGS__);     \
    if (E == 64 && F == 256) return NAME<64, 256>(__VA_ARGS__);     \
    if (E == 128 && F == 64) return NAME<128, 64>(__VA_ARGS__);     \
    if (E == 128 && F == 128) return NAME<128, 128>(__VA_ARGS__);   \
    if (E == 128 && F == 256) return NAME<128, 256>(__VA_ARGS__);   \
    if (E == 256 && F == 64) return NAME<256, 64>(__VA_ARGS__);     \
    if (E == 256 && F == 128) return NAME<256, 128>(__VA_ARGS__);   \
    if (E == 256 && F == 256) return NAME<256, 256>(__VA_ARGS__);   \
    return hipErrorInvalidValue;                                    \
  } while (0)

hipError_t la_launch(int E, int F, LaMode mode, bool bf16, const LaWalk& g, unsigned grid, hipStream_t stream) {
  SSS_LA_PICK(la_run, mode, bf16, g, grid, stream);
}
hipError_t la_launch_folds(int E, int F, bool bf16, const LaWalk& fwd, const LaWalk& rev, unsigned n, hipStream_t stream) {
  SSS_LA_PICK(la_run_folds, bf16, fwd, rev, n, stream);
}
hipError_t la_launch_grads(int E, int F, bool bf16, const LaWalk& dq, const LaWalk& dk, const LaWalk& dv, unsigned n,
                           hipStream_t stream) {
  SSS_LA_PICK(la_run_grads, bf16, dq, dk, dv, n, stream);
}
#undef SSS_LA_PICK

// One thread per element of the heads' states, over the segments in turn, the loads of sixteen at once (without
// regard to the flags, which come with them: where one is 0 nothing was written, and nothing is used).  Lanes of
// a wave whose elements are of one head share a decay.  blockIdx.y 1: backwards.  Bound by latency, a trip to
// memory per sixteen segments: both directions of 16 segments x 16 heads x 128 x 128 take 15 us (63 MB), of 32 segments
// x 6 x 64 x 50 8 us; with eight loads at once and a launch for each direction 34 (32 segments) and 20.
constexpr int kLaCarryBatch = 16;
static __global__ __launch_bounds__(256) void la_carry_kernel(LaCarry fwd, LaCarry back, int64_t hs, int H, int nseg) {
  const bool rev = blockIdx.y != 0;
  const float* const end = rev ? back.end : fwd.end;
  const float* const sum = rev ? back.sum : fwd.sum;
  const int32_t* const flag = rev ? back.flag : fwd.flag;
  float* const enter = rev ? back.enter : fwd.enter;
  const int64_t per = hs * H, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= per) return;
  const int h = (int)(i / hs), last = nseg - 1;  // segments 0 .. nseg - 2, or backwards nseg - 1 .. 1
  float v = 0.0f;
  for (int n0 = 0; n0 < last; n0 += kLaCarryBatch) {
    float e[kLaCarryBatch], d[kLaCarryBatch];
    int fl[kLaCarryBatch];
#pragma unroll
    for (int q = 0; q < kLaCarryBatch; ++q) {
      const int n = min(n0 + q, last - 1), c = rev ? last - n : n;
      fl[q] = flag[c];
      e[q] = end[c * per + i];
      d[q] = sum[(int64_t)c * H + h];
    }
#pragma unroll
    for (int q = 0; q < kLaCarryBatch; ++q) {
      if (n0 + q >= last || fl[q] == 0) continue;
      const int n = n0 + q;
      v = fl[q] == 2 ? e[q] : __builtin_fmaf(fast_exp2(d[q]), v, e[q]);
      enter[(int64_t)(rev ? last - n - 1 : n + 1) * per + i] = v;
    }
  }
}

hipError_t la_carry(const LaCarry& fwd, const LaCarry* rev, int64_t hs, int H, int nseg, hipStream_t stream) {
  hipLaunchKernelGGL(la_carry_kernel, dim3((unsigned)((hs * H + 255) / 256), rev != nullptr ? 2 : 1), dim3(256), 0, stream, fwd,
                     rev != nullptr ? *rev : fwd, hs, H, nseg);
  return hipGetLastError();
}

// dg_t, the sum over all pairs of tokens j < t <= i of their parts of the loss' gradient, tile by tile from the
// right.  Pairs in one tile come summed (within).  The others: with r = q dq from earlier tiles and c = k dk from
// later ones, those of a tile's own i are the r from t on, those of its own j the c before t, and those with both
// outside (through) the sum of r of all tiles to the right less that of c from the tile on.  The last tile of a
// segment's part of a sequence starts that sum with a `through` of its own, formed without a difference.  (Whole dq
// and dk would do as well, but roundings of pairs that cancel would be carried over the segment: 3e-5 of dg's norm in
// place of 3e-7.)  Nothing passes a token whose decay is a cut (kLaCut): its dg is zero, and so is a tile's `through` that
// has one, exactly, where the difference would leave roundings of however large sums behind it.  A wave per segment and head; the sums are 64-bit.  Bound by the latency of a wave's tiles in turn:
// 8192 tokens x 16 heads in 16 segments 10 us, 1001 x 6 in 32 4 us.
static __global__ __launch_bounds__(64) void la_finish_kernel(LaFinish a) {
  const int lane = threadIdx.x;
  const int h = (int)(blockIdx.x % (unsigned)a.H), seg = (int)(blockIdx.x / (unsigned)a.H);
  const int c0 = seg * a.K, tend = min(c0 + a.K, a.tokens);
  const LaBounds cu(a.cu, a.nseq, lane);
  const int lo = min(max(cu.at(0), 0), a.tokens), hi = min(max(cu.at(a.nseq), 0), a.tokens);
  const int64_t H = a.H;
  double sum = 0.0;
  auto clear = [&](int b, int e) {
    for (int t = b + lane; t < e; t += 64) {
      if (a.part == nullptr) a.dg[t * H + h] = 0.0f;
      if (a.dbeta != nullptr) a.dbeta[t * H + h] = 0.0f;
    }
  };
  int t = max(c0, lo);
  const int stop = min(tend, hi);
  const int gap = min(t, tend);
  clear(c0, gap);
  clear(max(max(stop, c0), gap), tend);
  int s = t < stop ? cu.find(t) : 0;
  while (t < stop) {
    const int end = min(cu.at(s + 1), hi);
    if (end <= t) {
      if (++s >= a.nseq) break;
      continue;
    }
    const int e = min(end, tend);
    double through = end > tend ? a.edge[seg * H + h] : a.last[s * H + h], x = 0.0;
    const int last = (e - t - 1) / a.tile;
    // a tile's values, asked for during the tile before (the decays, which lie apart, cost 2 us of 8192 tokens x 16 heads otherwise)
    float next[6];
    auto fetch = [&](int m) {
      const int at = min(t + a.tile * m + lane, e - 1);
      const int64_t p = (int64_t)h * a.tokens + at;
      next[0] = a.rows[p];
      next[1] = a.cols2[p];
      next[2] = a.within[p];
      next[3] = a.dbeta != nullptr ? a.cols[p] : 0.0f;
      next[4] = a.beta != nullptr ? a.beta[at * a.beta_st + h] : 1.0f;
      next[5] = a.g[at * a.g_st + h];
    };
    fetch(last);
    for (int m = last; m >= 0; --m) {
      const int at = t + a.tile * m + lane;
      const bool in = lane < a.tile && at < e, cut = in && next[5] <= kLaCut;
      const float r = in ? next[0] : 0.0f, w = next[2], c0 = next[1], k = next[3], c = in ? c0 * next[4] : 0.0f;
      if (m > 0) fetch(m - 1);
      if (in && a.dbeta != nullptr) a.dbeta[at * H + h] = k + c0;
      double rs = (double)r, cs = (double)c;  // from the lane on; up to the lane
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double up = __shfl_down(rs, d), dn = __shfl_up(cs, d);
        if (lane + d < 64) rs += up;
        if (lane >= d) cs += dn;
      }
      if (m != last) through = x - __shfl(cs, 63);
      if (__builtin_amdgcn_ballot_w64(cut) != 0) through = 0.0;
      x = through + __shfl(rs, 0);
      if (in) {
        const double v = cut ? 0.0 : through + rs + (cs - (double)c) + (double)w;
        if (a.part == nullptr) a.dg[at * H + h] = (float)v;
        else sum += v;
      }
    }
    t = e;
  }
  if (a.part != nullptr) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (lane == 0) a.part[seg * H + h] = (float)sum;
  }
}

static __global__ __launch_bounds__(256) void la_colsum_kernel(const float* __restrict__ part, float* __restrict__ out, int rows,
                                                               int64_t cols) {
  column_sums<8>(part, rows, cols, [=](int64_t col, float s) { out[col] = s; });
}

hipError_t la_finish(const LaFinish& a, hipStream_t stream) {
  if (a.nseg > 0) hipLaunchKernelGGL(la_finish_kernel, dim3((unsigned)(a.nseg * a.H)), dim3(64), 0, stream, a);
  if (a.part != nullptr)
    hipLaunchKernelGGL(la_colsum_kernel, dim3(colsum_blocks(a.H)), dim3(256), 0, stream, a.part, a.dg, a.nseg, (int64_t)a.H);
  if (a.dD != nullptr)
    hipLaunchKernelGGL(la_colsum_kernel, dim3(colsum_blocks(a.H)), dim3(256), 0, stream, a.trace, a.dD, a.nseg, (int64_t)a.H);
  return hipGetLastError();
}

// A thread per element, up to 2^30 threads: a launch counts them in 32 bits.
constexpr int64_t kLaSumBlocks = (int64_t)1 << 22;
template <bool BF16>
static __global__ __launch_bounds__(256) void la_sum_heads_kernel(LaSum a, LaSum b, int64_t tokens, int heads, int d) {
  const bool second = blockIdx.y != 0;
  const float* const part = second ? b.part : a.part;
  char* const out = (char*)(second ? b.out : a.out);
  const int rep = second ? b.rep : a.rep;
  const int64_t n = tokens * (heads / rep) * d;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {  // an element of out
    const int64_t row = i / d;
    const float* p = part + row * rep * d + (i - row * d);
    float s = 0.0f;
    for (int r = 0; r < rep; ++r) s += p[(int64_t)r * d];
    if constexpr (BF16) ((uint16_t*)out)[i] = (uint16_t)vec_bf16_pair(s, 0.0f);
    else ((float*)out)[i] = s;
  }
}

hipError_t la_sum_heads(const LaSum& a, const LaSum* b, int64_t tokens, int heads, int d, bool bf16, hipStream_t stream) {
  const int rep = b != nullptr ? std::min(a.rep, b->rep) : a.rep;
  const int64_t n = tokens * (heads / rep) * d;
  const dim3 grid((unsigned)std::min((n + 255) / 256, kLaSumBlocks), b != nullptr ? 2 : 1);
  if (bf16) hipLaunchKernelGGL(la_sum_heads_kernel<true>, grid, dim3(256), 0, stream, a, b != nullptr ? *b : a, tokens, heads, d);
  else hipLaunchKernelGGL(la_sum_heads_kernel<false>, grid, dim3(256), 0, stream, a, b != nullptr ? *b : a, tokens, heads, d);
  return hipGetLastError();
}

static __global__ __launch_bounds__(256) void la_empty_kernel(const int32_t* __restrict__ cu, const float* __restrict__ dfinal,
                                                              float* __restrict__ dinitial, int nseq, int tokens, int64_t per) {
  const int lo = min(max(cu[0], 0), tokens), hi = min(max(cu[nseq], 0), tokens);
  for (int64_t s = blockIdx.x; s < nseq; s += gridDim.x) {
    if (min(cu[s + 1], hi) > max(cu[s], lo)) continue;
    for (int64_t i = threadIdx.x; i < per; i += 256) dinitial[s * per + i] = dfinal != nullptr ? dfinal[s * per + i] : 0.0f;
  }
}

hipError_t la_empty(const int32_t* cu, const float* dfinal, float* dinitial, int nseq, int tokens, int64_t per, hipStream_t stream) {
  hipLaunchKernelGGL(la_empty_kernel, dim3((unsigned)std::min(nseq, 1 << 22)), dim3(256), 0, stream, cu, dfinal, dinitial, nseq, tokens, per);
  return hipGetLastError();
}

// One token of each row: S <- e^g S + beta k v^T in its slot, o = scale q S + D v.  A workgroup takes a row
// and head: V adjacent columns and every RL-th row of S per thread, eight loads in flight.  Bound by the
// states, read once and written once: 256 rows x 80 heads x 128 x 64, 1342 MB, 249 us (5.4 TB/s); of 3 rows x 16 heads
// of 64 x 64 4 us, a launch and two trips to memory.
template <bool BF16>
__device__ __forceinline__ float la_get(const char* p, int64_t i) {
  if constexpr (BF16) return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
  else return ((const float*)p)[i];
}

template <bool BF16, int V, int CG>
static __global__ __launch_bounds__(256) void la_step_kernel(LaStep a) {
  constexpr int RL = 256 / CG, ES = BF16 ? 2 : 4;
  constexpr int G = CG < 64 ? 4 : RL;  // partial sums of an output
  __shared__ float lq[256], lk[256], lo[G * CG * V];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / (unsigned)a.H;
  const int h = (int)(blockIdx.x - (unsigned)b * (unsigned)a.H);
  const int dk = a.q.width, dv = a.v.width;
  const int c = (tid % CG) * V, rl = tid / CG;
  const int slot = a.sidx != nullptr ? a.sidx[b] : (int)b;
  const bool kept = (unsigned)slot < (unsigned)a.slots, in = c < dv;
  float* const S = kept ? a.state + ((int64_t)slot * a.H + h) * dk * dv + c : nullptr;
  constexpr int B = 8;
  Vec<false, V> s[B];
  auto load = [&](int e0) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = e0 + i * RL;
      if (kept && in && e < dk) s[i].template load<true>(S + (int64_t)e * dv);
      else s[i].zero();
    }
  };
  load(rl);
  if (tid < dk) {
    const char* const q = a.q.p + ((h / a.q.rep) * a.q.sh + b * a.q.st) * ES;
    const char* const k = a.k.p + ((h / a.k.rep) * a.k.sh + b * a.k.st) * ES;
    lq[tid] = la_get<BF16>(q, tid) * a.scale;
    lk[tid] = la_get<BF16>(k, tid) * (a.beta != nullptr ? a.beta[b * a.beta_st + h] : 1.0f);
  }
  const float gv = a.g[b * a.g_st + h];
  const float decay = fast_exp2((float)((double)(gv < kLaCut ? kLaCut : gv) * 1.4426950408889634074));
  const char* const vp = a.v.p + ((h / a.v.rep) * a.v.sh + b * a.v.st) * ES;
  float v[V], o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = in ? la_get<BF16>(vp, c + i) : 0.0f;
    o[i] = 0.0f;
  }
  __syncthreads();
  for (int e0 = rl; e0 < dk; e0 += B * RL) {
    if (e0 != rl) load(e0);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = e0 + i * RL;
      if (e >= dk) continue;
      const float kk = lk[e], qq = lq[e];
      float n[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        n[j] = __builtin_fmaf(decay, s[i].get(j), kk * v[j]);
        o[j] = __builtin_fmaf(qq, n[j], o[j]);
      }
      if (kept && in) {
        Vec<false, V> r;
        r.set(n);
        r.template store<true>(S + (int64_t)e * dv);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int d = CG; d < 64; d *= 2) o[j] += __shfl_xor(o[j], d);
    if (CG >= 64 || (tid & 63) < CG) lo[(CG < 64 ? tid / 64 : rl) * (CG * V) + c + j] = o[j];
  }
  __syncthreads();
  for (int f = tid; f < dv; f += 256) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < G; ++i) r += lo[i * (CG * V) + f];
    if (a.D != nullptr) r += a.D[h] * la_get<BF16>(vp, f);
    const int64_t at = (b * a.H + h) * dv + f;
    if constexpr (BF16) ((uint16_t*)a.out)[at] = (uint16_t)vec_bf16_pair(r, 0.0f);
    else ((float*)a.out)[at] = r;
  }
}

template <bool BF16>
static hipError_t la_step_of(const LaStep& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.rows * a.H));
  const int dv = a.v.width;
#define SSS_LA_STEP(V, CG) hipLaunchKernelGGL((la_step_kernel<BF16, V, CG>), grid, dim3(256), 0, stream, a)
  if (dv % 4 == 0) {  // 16 adjacent bytes per lane
    if (dv <= 64) SSS_LA_STEP(4, 16);
    else if (dv <= 128) SSS_LA_STEP(4, 32);
    else SSS_LA_STEP(4, 64);
  } else {
    if (dv <= 64) SSS_LA_STEP(1, 64);
    else if (dv <= 128) SSS_LA_STEP(1, 128);
    else SSS_LA_STEP(1, 256);
  }
#undef SSS_LA_STEP
  return hipGetLastError();
}

hipError_t la_step(const LaStep& a, bool bf16, hipStream_t stream) {
  return bf16 ? la_step_of<true>(a, stream) : la_step_of<false>(a, stream);
}

}  // namespace sss

// packed_conv.hip -- gfx950 kernels of the causal depthwise convolution for serving: packed
// prompts of any lengths with the inputs before them in a cache, and the single-token step.
//
// Per sequence and channel d, with u = x inside the sequence and, before it, the W-1 inputs
// that the sequence's cache slot keeps (zero where there are none):
//   out[t,d] = bias[d] + sum_{k<W} w[d,k] * u[t-(W-1)+k, d],  then optionally silu,
// and the slot is left with the last W-1 inputs.  Pure streaming: 2 + 2 bytes per element in
// bf16 and W fmas.
#include "vec.h"
#include "kernels.h"

#include <algorithm>

namespace sss {

constexpr int kPConvU = 2;  // steps per load batch (4 and 8 measured within 1%)

struct PConvGeo {
  int64_t x_stride;  // elements between tokens of x
  int tokens, nseq, slots, D, K, ngroups;
};

// One wave = 64 lanes x CPL adjacent channels and one chunk of K tokens of the packed axis, cut
// without regard to the sequences (whose lengths only the device knows).  The wave walks the
// sequences of its chunk; inside one, the last W-1 inputs stay in registers as a sliding
// window.  The first W-1 tokens of a sequence belong to the chunk that holds its start, also
// where they pass the chunk's end: only that wave reads the sequence's cache slot, before it
// writes the new contents, so that the slot is updated in place without a second launch.
// RAGGED: CPL does not divide the channels.
template <int W, bool BF16, bool SILU, int CPL, bool RAGGED>
__global__ __launch_bounds__(64) void packed_conv_kernel(const char* __restrict__ x, const float* __restrict__ w,
                                                         const float* __restrict__ bias, char* __restrict__ state,
                                                         const int32_t* __restrict__ cu,
                                                         const int32_t* __restrict__ sidx,
                                                         const uint8_t* __restrict__ init, char* __restrict__ out,
                                                         PConvGeo g) {
  using R = Vec<BF16, CPL>;
  constexpr int ES = R::ES;
  const int lane = threadIdx.x;
  const uint32_t lid = xcd_remap(blockIdx.x, gridDim.x);
  const int grp = (int)(lid % (uint32_t)g.ngroups);
  const int c0 = (int)(lid / (uint32_t)g.ngroups) * g.K;
  const int d0 = grp * 64 * CPL;
  // The lane at the row's end takes its last CPL channels and stores only those that the lane
  // before it does not have: another wave may have those, and the slots are updated in place.
  const int dc = min(d0 + lane * CPL, g.D - CPL);
  const int skip = RAGGED ? min(d0 + lane * CPL - dc, CPL) : 0;
  const int64_t D = g.D;

  const int lo = max(cu[0], 0), hi = min(cu[g.nseq], g.tokens);
  int t = max(c0, lo);
  const int tend = min(c0 + g.K, hi);
  if (t >= tend) return;
  int s = min(max(find_seq(cu, g.nseq, t, lane), 0), g.nseq - 1);
  if (d0 + lane * CPL >= g.D) return;  // (the search takes the whole wave)

  float wk[CPL][W], bv[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) wk[c][k] = w[(int64_t)(dc + c) * W + k];
    bv[c] = bias != nullptr ? bias[dc + c] : 0.0f;
  }
  const int64_t xrow = g.x_stride * ES, orow = D * ES;
  const uint32_t lo_ = (uint32_t)dc * ES;  // the lane's bytes in a row
  const char* const xl = x + lo_;

  while (t < tend) {
    const int end = min(cu[s + 1], hi);
    if (end <= t) {  // past this sequence (or an empty one)
      if (++s >= g.nseq) break;
      continue;
    }
    const int beg = min(max(cu[s], 0), t);
    if (beg < c0 && t - beg < W - 1) {  // the chunk before this one has these tokens
      t = min(beg + W - 1, end);
      continue;
    }
    const int e = min(end, beg < c0 ? tend : max(tend, beg + W - 1));
    const int slot = sidx != nullptr ? sidx[s] : s;
    const bool kept = state != nullptr && (unsigned)slot < (unsigned)g.slots;

    // the W-1 inputs before t: of the sequence, or of its slot where t is its first token
    R hist[W > 1 ? W - 1 : 1];
    if (t > beg) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) hist[k].load(xl + (int64_t)(t - (W - 1) + k) * xrow);
    } else {
      char* const sl = state + ((int64_t)slot * (W - 1) * D + dc) * ES;
      const bool started = kept && init != nullptr && init[s] != 0;
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        if (started) hist[k].load(sl + (int64_t)k * D * ES);
        else hist[k].zero();
      }
      if (kept) {  // the last W-1 of (history, tokens)
        const int len = end - beg;
        R nw[W > 1 ? W - 1 : 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          const int p = len + k - (W - 1);  // position in the sequence; negative: history
          if (p >= 0) {
            nw[k].load(xl + (int64_t)(beg + p) * xrow);
          } else {
            nw[k] = hist[k];
#pragma unroll
            for (int j = k + 1; j < W - 1; ++j)
              if (k + len == j) nw[k] = hist[j];
          }
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) nw[k].store_from(sl + (int64_t)k * D * ES, skip);
      }
    }
    float win[CPL][W];
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int k = 0; k < W - 1; ++k) win[c][k] = hist[k].get(c);

    const int len = e - t;
    const char* const xb = x + (int64_t)t * xrow;
    char* const ob = out + (int64_t)t * orow;
    R q[2][kPConvU];
    auto load = [&](int slot_, int t0) {
#pragma unroll
      for (int i = 0; i < kPConvU; ++i)
        q[slot_][i].template load<true>(row_at(xb, (int64_t)min(t0 + i, len - 1) * xrow), lane_at(lo_));
    };
    auto step = [&](const R& in, int i) {
      float o[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        win[c][W - 1] = in.get(c);
        float v = bv[c];
#pragma unroll
        for (int k = 0; k < W; ++k) v = __builtin_fmaf(wk[c][k], win[c][k], v);
        o[c] = SILU ? silu(v) : v;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[c][k] = win[c][k + 1];
      }
      R r;
      r.set(o);
      // non-temporal both ways: 75 us on 16384 x 5120 (4.5 TB/s), 78 with cached stores, 79 with
      // cached loads
      if constexpr (RAGGED) r.template store_from<true>(row_at(ob, (int64_t)i * orow), lane_at(lo_), skip);
      else r.template store<true>(row_at(ob, (int64_t)i * orow), lane_at(lo_));
    };
    load(0, 0);
    int t0 = 0;
    for (; t0 + 2 * kPConvU <= len; t0 += 2 * kPConvU) {
      load(1, t0 + kPConvU);
#pragma unroll
      for (int i = 0; i < kPConvU; ++i) step(q[0][i], t0 + i);
      load(0, t0 + 2 * kPConvU);
#pragma unroll
      for (int i = 0; i < kPConvU; ++i) step(q[1][i], t0 + kPConvU + i);
    }
    if (t0 < len) {
      load(1, t0 + kPConvU);
#pragma unroll
      for (int i = 0; i < kPConvU; ++i)
        if (t0 + i < len) step(q[0][i], t0 + i);
#pragma unroll
      for (int i = 0; i < kPConvU; ++i)
        if (t0 + kPConvU + i < len) step(q[1][i], t0 + kPConvU + i);
    }
    t = e;
  }
}

// The single-token step: one thread per row and CPL channels reads the slot's W-1 inputs and
// the new one, writes the output and the slot shifted by one.  A row without a slot (a negative
// index) starts from zeros and keeps nothing.
template <int W, bool BF16, int CPL>
__global__ __launch_bounds__(256) void conv_update_kernel(const char* __restrict__ x, const float* __restrict__ w,
                                                          const float* __restrict__ bias, char* __restrict__ state,
                                                          const int32_t* __restrict__ sidx, char* __restrict__ out,
                                                          int64_t x_stride, int rows, int slots, int D, int bpr,
                                                          int apply_silu) {
  using R = Vec<BF16, CPL>;
  constexpr int ES = R::ES;
  const int row = (int)(blockIdx.x / (unsigned)bpr);
  const int li = (int)(blockIdx.x - (unsigned)row * bpr) * (int)blockDim.x + (int)threadIdx.x;
  const int dl = li * CPL;
  if (dl >= D) return;
  // as above: the last thread of a row that CPL does not divide stores only its own channels
  const int dc = min(dl, D - CPL);
  const int skip = dl - dc;
  const int slot = sidx != nullptr ? sidx[row] : row;
  const bool kept = (unsigned)slot < (unsigned)slots;
  char* const sl = state + ((int64_t)slot * (W - 1) * D + dc) * ES;
  R in, hist[W > 1 ? W - 1 : 1];
  in.load(x + ((int64_t)row * x_stride + dc) * ES);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    if (kept) hist[k].load(sl + (int64_t)k * D * ES);
    else hist[k].zero();
  }
  float o[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    float v = bias != nullptr ? bias[dc + c] : 0.0f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) v = __builtin_fmaf(w[(int64_t)(dc + c) * W + k], hist[k].get(c), v);
    v = __builtin_fmaf(w[(int64_t)(dc + c) * W + W - 1], in.get(c), v);
    o[c] = apply_silu ? silu(v) : v;
  }
  R r;
  r.set(o);
  r.store_from(out + ((int64_t)row * D + dc) * ES, skip);
  if (kept) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      (k + 1 < W - 1 ? hist[k + 1 < W - 1 ? k + 1 : 0] : in).store_from(sl + (int64_t)k * D * ES, skip);
  }
}

template <bool BF16>
constexpr int kPConvCpl = BF16 ? 4 : 2;  // 8 bytes per lane

static int chunk_tokens(int64_t tokens, int64_t groups, int width, int num_cus) {
  // Short-lived waves stream best: 40 per CU (16384 x 5120: 75 us, chunks of 32 tokens; 76 with 20
  // or 80).  Chunks of 12 tokens at least, of 8 where those leave less than eight waves per CU
  // (16384 x 1024: 20.0 us with 12, 20.9 with 8, 22.5 with 32; 512 x 2048: 5.3 us with 8, 6.0 with
  // 12, 9.0 with 32).
  const int64_t cus = std::max(num_cus, 1);
  const int64_t chunks = std::max<int64_t>(1, cus * 40 / std::max<int64_t>(1, groups));
  const int64_t least = groups * ((tokens + 7) / 8) < cus * 8 ? 8 : 12;
  int64_t k = std::max<int64_t>((tokens + chunks - 1) / chunks, least);
  const int forced = env_int("SSS_FORCE_SEGMENTS", 0);
  if (forced > 0) k = std::max<int64_t>((tokens + forced - 1) / forced, width);
  return (int)std::max<int64_t>(k, width);  // a sequence's first width-1 tokens reach one chunk further at most
}

template <int W, bool BF16, bool SILU, int CPL, bool RAGGED>
static hipError_t run_packed(const PackedConvArgs& a, int num_cus, hipStream_t stream) {
  PConvGeo g{};
  g.x_stride = a.x_stride;
  g.tokens = (int)a.tokens;
  g.nseq = (int)a.nseq;
  g.slots = (int)a.slots;
  g.D = (int)a.dim;
  g.ngroups = (int)((a.dim + 64 * CPL - 1) / (64 * CPL));
  g.K = chunk_tokens(a.tokens, g.ngroups, W, num_cus);
  const int64_t chunks = (a.tokens + g.K - 1) / g.K;
  hipLaunchKernelGGL((packed_conv_kernel<W, BF16, SILU, CPL, RAGGED>), dim3((unsigned)(chunks * g.ngroups)), dim3(64), 0, stream,
                     (const char*)a.x, a.w, a.bias, (char*)a.state, a.cu, a.sidx, a.init, (char*)a.out, g);
  return hipGetLastError();
}

template <int W, bool BF16, int CPL>
static hipError_t run_step(const PackedConvArgs& a, hipStream_t stream) {
  const int lanes = (int)((a.dim + CPL - 1) / CPL);
  const int bpr = (lanes + 255) / 256;
  hipLaunchKernelGGL((conv_update_kernel<W, BF16, CPL>), dim3((unsigned)(a.tokens * bpr)), dim3(256), 0, stream,
                     (const char*)a.x, a.w, a.bias, (char*)a.state, a.sidx, (char*)a.out, a.x_stride, (int)a.tokens,
                     (int)a.slots, (int)a.dim, bpr, a.silu);
  return hipGetLastError();
}

template <int W, bool BF16, bool SILU>
static hipError_t run_prompts(const PackedConvArgs& a, int num_cus, hipStream_t stream) {
  constexpr int kWide = kPConvCpl<BF16>;
  if (a.dim < kWide) return run_packed<W, BF16, SILU, 1, false>(a, num_cus, stream);
  return a.dim % kWide == 0 ? run_packed<W, BF16, SILU, kWide, false>(a, num_cus, stream)
                            : run_packed<W, BF16, SILU, kWide, true>(a, num_cus, stream);
}

template <int W, bool BF16>
static hipError_t run_width(const PackedConvArgs& a, int num_cus, hipStream_t stream) {
  constexpr int kWide = kPConvCpl<BF16>;
  if (a.step) return a.dim >= kWide ? run_step<W, BF16, kWide>(a, stream) : run_step<W, BF16, 1>(a, stream);
  return a.silu ? run_prompts<W, BF16, true>(a, num_cus, stream) : run_prompts<W, BF16, false>(a, num_cus, stream);
}

template <bool BF16>
static hipError_t run_type(const PackedConvArgs& a, int num_cus, hipStream_t stream) {
  switch (a.width) {
    case 1: return run_width<1, BF16>(a, num_cus, stream);
    case 2: return run_width<2, BF16>(a, num_cus, stream);
    case 3: return run_width<3, BF16>(a, num_cus, stream);
    case 4: return run_width<4, BF16>(a, num_cus, stream);
    case 5: return run_width<5, BF16>(a, num_cus, stream);
    case 6: return run_width<6, BF16>(a, num_cus, stream);
    case 7: return run_width<7, BF16>(a, num_cus, stream);
    case 8: return run_width<8, BF16>(a, num_cus, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_packed_conv(const PackedConvArgs& a, int num_cus, hipStream_t stream) {
  return a.bf16 ? run_type<true>(a, num_cus, stream) : run_type<false>(a, num_cus, stream);
}

}  // namespace sss

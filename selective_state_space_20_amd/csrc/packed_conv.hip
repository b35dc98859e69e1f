// packed_conv.hip -- gfx950 kernels of the causal depthwise convolution for serving: packed
// prompts of any lengths with the inputs before them in a cache, and the single-token step.
//
// Per sequence and channel d, with u = x inside the sequence and, before it, the W-1 inputs
// that the sequence's cache slot keeps (zero where there are none):
//   out[t,d] = bias[d] + sum_{k<W} w[d,k] * u[t-(W-1)+k, d],  then optionally silu,
// and the slot is left with the last W-1 inputs.  Pure streaming: 2 + 2 bytes per element in
// bf16 and W fmas.
#include "seq_walk.h"
#include "vec.h"
#include "kernels.h"

namespace sss {

constexpr int kPConvK = 8;      // tokens per chunk
constexpr int kPConvWaves = 4;  // chunks per workgroup, one per wave

struct PConvGeo {
  int64_t x_stride;  // elements between tokens of x
  int tokens, nseq, slots, D, ngroups;
};

// One wave = 64 lanes x CPL adjacent channels (16 or 8 bytes) and one chunk of 8 tokens of the
// packed axis, cut without regard to the sequences, whose lengths only the device knows.  It loads
// its rows and the W-1 before them all at once and, where they lie inside one sequence, computes
// and stores them without a loop: nothing in flight waits for anything, and the W-1 shared
// rows come from the L2 of the XCD that the chunks next to each other run on (they alone are
// read through the caches).  Bound by memory: 16384 x 5120 bf16 takes 61-65 us (336 MB, 5.2-5.5
// TB/s, where a plain copy reaches 5.3); waves that walk 32 or 64 rows, two to eight at a time, 73.
//
// A chunk in which a sequence starts or ends, or has just started, is walked token by token.
// The first W-1 tokens of a sequence belong to the chunk that holds its start, also where they
// pass the chunk's end: only that wave reads the sequence's cache slot, before it writes the new
// contents, so that the slot is updated in place without a second launch.
// RAGGED: CPL does not divide the channels.
template <int W, bool BF16, bool SILU, int CPL, bool RAGGED>
__global__ __launch_bounds__(64 * kPConvWaves) void packed_conv_kernel(const char* __restrict__ x, const float* __restrict__ w,
                                                         const float* __restrict__ bias, char* __restrict__ state,
                                                         const int32_t* __restrict__ cu,
                                                         const int32_t* __restrict__ sidx,
                                                         const uint8_t* __restrict__ init, char* __restrict__ out,
                                                         PConvGeo g) {
  using R = Vec<BF16, CPL>;
  constexpr int ES = R::ES, K = kPConvK, H = W - 1;
  static_assert(H <= K, "a sequence's first W-1 tokens reach one chunk further at most");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t lid = xcd_remap(blockIdx.x, gridDim.x);
  const int grp = (int)(lid % (uint32_t)g.ngroups);
  const int c0 = ((int)(lid / (uint32_t)g.ngroups) * kPConvWaves + wave) * K;
  const int d0 = grp * 64 * CPL;
  // The lane at the row's end takes its last CPL channels and stores only those that the lane
  // before it does not have: another wave may have those, and the slots are updated in place.
  // Lanes past it load the same and leave after the search, which takes the whole wave.
  const int dc = min(d0 + lane * CPL, g.D - CPL);
  const int skip = RAGGED ? min(d0 + lane * CPL - dc, CPL) : 0;
  const int64_t D = g.D;
  const int64_t xrow = g.x_stride * ES, orow = D * ES;
  const uint32_t at = (uint32_t)dc * ES;  // the lane's bytes in a row

  const SeqSearch search(cu, g.nseq, lane);
  const int lo = max(cu[0], 0), hi = min(cu[g.nseq], g.tokens);
  R q[K + H];
  auto load_rows = [&]() {
#pragma unroll
    for (int i = 0; i < K + H; ++i) {
      const row_ptr r = row_at(x, (int64_t)min(max(c0 - H + i, 0), g.tokens - 1) * xrow);
      if (i >= H && i < K) q[i].template load<true>(r, lane_at(at));
      else q[i].load(r, lane_at(at));
    }
  };
  // A lane's CPL * W weights are adjacent, so that loads of its own would take 64 cache lines
  // each: the workgroup, four chunks of the same channels, loads them once in whole lines and
  // turns them round in LDS, lanes an odd number of 16-byte pieces apart (16384 x 5120: 66 us; 92
  // with loads of each lane's own, 74 with a turn in every wave).
  constexpr int P = CPL * W / 4;  // 16-byte pieces per lane
  constexpr bool kTurn = CPL >= 4;
  __shared__ float wlds[kTurn ? 64 * (P | 1) * 4 : 1];
  float wk[CPL][W], bv[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) bv[c] = bias != nullptr ? bias[dc + c] : 0.0f;
  if (kTurn && d0 + 64 * CPL <= g.D) {
    const float* const wg = w + (int64_t)d0 * W;
    constexpr int kPer = kTurn ? (64 * P + 64 * kPConvWaves - 1) / (64 * kPConvWaves) : 1;
    Vec<false, 4> piece[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) piece[j].load(wg + min(j * 64 * kPConvWaves + (int)threadIdx.x, 64 * P - 1) * 4);
    load_rows();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = j * 64 * kPConvWaves + (int)threadIdx.x, l = i / (kTurn ? P : 1);
      float* const to = wlds + (l * (P | 1) + i - l * P) * 4;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i < 64 * P) to[c] = piece[j].get(c);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CPL * W; ++i) wk[i / W][i % W] = wlds[lane * (P | 1) * 4 + i];
  } else {
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int k = 0; k < W; ++k) wk[c][k] = w[(int64_t)(dc + c) * W + k];
    load_rows();
  }
  int t = max(c0, lo);
  const int tend = min(c0 + K, hi);
  if (t >= tend) return;
  int s = min(max(search.find(t), 0), g.nseq - 1);
  if (d0 + lane * CPL >= g.D) return;

  auto put = [&](const R& r, int64_t token) {
    const row_ptr p = row_at(out, token * orow);
    if constexpr (RAGGED) r.template store_from<true>(p, lane_at(at), skip);
    else r.template store<true>(p, lane_at(at));
  };
  if (tend - t == K && began_before(cu[s], c0 - H + 1) && cu[s + 1] >= tend) {
    R o[K];
#pragma unroll
    for (int c = 0; c < CPL; c += 2) {
      float v[2][K];
#pragma unroll
      for (int h = 0; h < 2 && c + h < CPL; ++h) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
          float a = bv[c + h];
#pragma unroll
          for (int k = 0; k < W; ++k) a = __builtin_fmaf(wk[c + h][k], q[i + k].get(c + h), a);
          v[h][i] = SILU ? silu(a) : a;
        }
      }
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if constexpr (BF16) {
          o[i].w[c >> 1] = vec_bf16_pair(v[0][i], CPL > 1 ? v[1][i] : 0.0f);
        } else {
          o[i].w[c] = __builtin_bit_cast(uint32_t, v[0][i]);
          if constexpr (CPL > 1) o[i].w[c + 1] = __builtin_bit_cast(uint32_t, v[1][i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) put(o[i], c0 + i);
    return;
  }

  const char* const xl = x + at;
  while (t < tend) {
    const int end = min(cu[s + 1], hi);
    if (end <= t) {  // past this sequence (or an empty one)
      if (++s >= g.nseq) break;
      continue;
    }
    const ConvPiece piece = conv_piece(cu[s], end, t, c0, tend, H);
    if (!piece.mine) {
      t = piece.next;
      continue;
    }
    const int beg = piece.beg, e = piece.next;
    const int slot = sidx != nullptr ? sidx[s] : s;
    const bool kept = state != nullptr && (unsigned)slot < (unsigned)g.slots;

    // the W-1 inputs before t: of the sequence, or of its slot where t is its first token
    R hist[W > 1 ? H : 1];
    if (t > beg) {
#pragma unroll
      for (int k = 0; k < H; ++k) hist[k].load(xl + (int64_t)(t - H + k) * xrow);
    } else {
      char* const sl = state + ((int64_t)slot * H * D + dc) * ES;
      const bool started = kept && init != nullptr && init[s] != 0;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        if (started) hist[k].load(sl + (int64_t)k * D * ES);
        else hist[k].zero();
      }
      if (kept) {  // the last W-1 of (history, tokens)
        const int len = end - beg;
        R nw[W > 1 ? H : 1];
#pragma unroll
        for (int k = 0; k < H; ++k) {
          const int p = len + k - H;  // position in the sequence; negative: history
          if (p >= 0) {
            nw[k].load(xl + (int64_t)(beg + p) * xrow);
          } else {
            nw[k] = hist[k];
#pragma unroll
            for (int j = k + 1; j < H; ++j)
              if (k + len == j) nw[k] = hist[j];
          }
        }
#pragma unroll
        for (int k = 0; k < H; ++k) nw[k].store_from(sl + (int64_t)k * D * ES, skip);
      }
    }
    float win[CPL][W];
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int k = 0; k < H; ++k) win[c][k] = hist[k].get(c);
    auto step = [&](const R& cur) {
      float o[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        win[c][W - 1] = cur.get(c);
        float v = bv[c];
#pragma unroll
        for (int k = 0; k < W; ++k) v = __builtin_fmaf(wk[c][k], win[c][k], v);
        o[c] = SILU ? silu(v) : v;
#pragma unroll
        for (int k = 0; k < H; ++k) win[c][k] = win[c][k + 1];
      }
      R r;
      r.set(o);
      put(r, t);
    };
    // The chunk's tokens are in registers, those after it are not.  Two loops: in one that takes each
    // token from either, the compiler (ROCm 7.2.0) lost a copy of the window in every fp32 kernel of
    // 8 bytes per lane and three taps or more.  Of a row's two registers, set by a select or by a load, it
    // took the upper one for undefined at the loop's head, and dropped `window = the next` of the
    // lane's second channel.  tests/test_codegen.py looks for such copies in the machine code.
    for (const int last = min(e, c0 + K); t < last; ++t) {
      R cur = q[H];
#pragma unroll
      for (int i = 1; i < K; ++i)
        if (t - c0 == i) cur = q[H + i];
      step(cur);
    }
    for (; t < e; ++t) {
      R cur;
      cur.load(xl + (int64_t)t * xrow);
      step(cur);
    }
  }
}

// The single-token step: one thread per row and CPL channels reads the slot's W-1 inputs and
// the new one, writes the output and the slot shifted by one.  A row without a slot (a negative
// index) starts from zeros and keeps nothing.  4 rows x 5120 take 3 us, one trip to memory; the call
// takes 10, of which the host's part is the rest.
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

template <int W, bool BF16, bool SILU, int CPL, bool RAGGED>
static hipError_t run_packed(const PackedConvArgs& a, hipStream_t stream) {
  PConvGeo g{};
  g.x_stride = a.x_stride;
  g.tokens = (int)a.tokens;
  g.nseq = (int)a.nseq;
  g.slots = (int)a.slots;
  g.D = (int)a.dim;
  g.ngroups = (int)((a.dim + 64 * CPL - 1) / (64 * CPL));
  const int64_t blocks = (a.tokens + kPConvK * kPConvWaves - 1) / (kPConvK * kPConvWaves);
  hipLaunchKernelGGL((packed_conv_kernel<W, BF16, SILU, CPL, RAGGED>), dim3((unsigned)(blocks * g.ngroups)), dim3(64 * kPConvWaves), 0, stream,
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

template <int W, bool BF16, bool SILU, int CPL>
static hipError_t run_ragged(const PackedConvArgs& a, hipStream_t stream) {
  return a.dim % CPL == 0 ? run_packed<W, BF16, SILU, CPL, false>(a, stream)
                          : run_packed<W, BF16, SILU, CPL, true>(a, stream);
}

template <int W, bool BF16, bool SILU>
static hipError_t run_prompts(const PackedConvArgs& a, hipStream_t stream) {
  // 16 bytes per lane stream best, 8 bytes have twice the waves, each with half the work: from
  // 64 MiB on the former (16384 x 5120 bf16: 66 us, 70 with 8 bytes), below it the latter
  // (16384 x 1024: 18.7 us, 19.8 with 16; 2000 x 5120: 13.5, 16.1; 64 x 5120: 6.5, 8.5)
  constexpr int kWide = BF16 ? 8 : 4;
  const bool large = a.tokens * a.dim * (BF16 ? 2 : 4) >= (int64_t)64 << 20;
  if (a.dim < kWide / 2) return run_packed<W, BF16, SILU, 1, false>(a, stream);
  return large && a.dim >= kWide ? run_ragged<W, BF16, SILU, kWide>(a, stream)
                                 : run_ragged<W, BF16, SILU, kWide / 2>(a, stream);
}

template <int W, bool BF16>
static hipError_t run_width(const PackedConvArgs& a, hipStream_t stream) {
  constexpr int kWide = BF16 ? 4 : 2;  // the step: 8 bytes per lane
  if (a.step) return a.dim >= kWide ? run_step<W, BF16, kWide>(a, stream) : run_step<W, BF16, 1>(a, stream);
  return a.silu ? run_prompts<W, BF16, true>(a, stream) : run_prompts<W, BF16, false>(a, stream);
}

template <bool BF16>
static hipError_t run_type(const PackedConvArgs& a, hipStream_t stream) {
  switch (a.width) {
    case 1: return run_width<1, BF16>(a, stream);
    case 2: return run_width<2, BF16>(a, stream);
    case 3: return run_width<3, BF16>(a, stream);
    case 4: return run_width<4, BF16>(a, stream);
    case 5: return run_width<5, BF16>(a, stream);
    case 6: return run_width<6, BF16>(a, stream);
    case 7: return run_width<7, BF16>(a, stream);
    case 8: return run_width<8, BF16>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_packed_conv(const PackedConvArgs& a, hipStream_t stream) {
  return a.bf16 ? run_type<true>(a, stream) : run_type<false>(a, stream);
}

}  // namespace sss

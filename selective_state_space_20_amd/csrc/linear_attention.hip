// linear_attention.hip -- gfx950 kernels of linear attention with a decay for each head, over packed
// sequences: outputs and gradients.  With log decays g_t <= 0 and input weights b_t,
//   S_t = e^(g_t) S_(t-1) + b_t k_t v_t^T,   o_t = scale q_t S_t + D v_t
// and for a loss with gradients do_t, the adjoint of the state runs backwards in time:
//   R_t = scale q_t do_t^T + e^(g_(t+1)) R_(t+1)
//   dq_t = scale S_t do_t,  dk_t = b_t R_t v_t,  dv_t = b_t R_t^T k_t + D do_t
//   db_t = k_t R_t v_t,     dg_t = <R_t, e^(g_t) S_(t-1)> = q_t dq_t - k_t dk_t + dg_(t+1)
//
// All of them are one walk in tiles of C tokens with a state M (E x F) in the accumulators of the
// matrix cores, G the sums of g from the tile's first token on:
//   out_i = sum_j e^(|G_i - G_j|) (x_i . y_j) z_j  +  e^(G_i) x_i M,   M <- e^(G_C) M + sum_j e^(G_C - G_j) y_j z_j^T
//            walk         x   y   z    M
//   outputs  forwards     q   k   v    S
//   dq       forwards     do  v   k    S^T
//   dk       backwards    v   do  q    R^T  (j >= i, and e^(G_C - G_i), e^(G_j) for the two weights)
//   dv       backwards    k   q   do   R
// The scores of a tile go through LDS once; M never leaves the registers of the wave that has its columns: a wave's
// accumulators of two 16-row tiles are, in parts, the operand of 32 rows of the next product as they lie.
//
// The packed axis is cut in segments of K tokens, whatever the sequences; a workgroup takes one
// segment and head.  The state that enters a segment comes from a first pass (kLaFold*: the update of M
// alone, for the one sequence that runs across the segment's edge) and a sum over the segments.
//
// Sums, decays (64-bit) and M are fp32 or more, and no operand that is formed here is rounded to one bf16.  What ends in
// bf16 results takes the scores and M (the outputs, dv), and dv's walk the weighted z, as the sum of two bf16 parts: 16
// bits, so that a bf16 result is a value in fp32 precision, rounded once.  (One part each left 0.0024 of the results' norm
// in place of the rounding's own 0.0017; prompts of 16384 x 80 x 128 x 64 took 325 us, of 32768 x 16 x 128 x 128 245, the
// gradients below 229.)  What goes into fp32 results (the states, and the parts of dg, db that come from other tiles)
// takes M and the weighted z as the sum of three, 24 bits of them.  Two parts in dq and dk would save 4%
// (301 -> 289 us of the gradients below, as they were) and leave 6e-6 of dg's norm instead of 3e-7.
//
// What bounds it.  The bytes are few (16384 tokens x 80 heads of 128 x 64: 449 MB, 85 us at a copy's rate) and so is
// the arithmetic (0.15 TFLOP with the extra parts, 120 us at a large product's rate); what is left is the chain of a
// tile: loads to LDS, barrier, scores, barrier, the products that need them and M, with two workgroups of four waves
// per CU (LDS and the registers of M) to fill each other's gaps.  So a tile is as long as LDS allows, its loads are
// in flight during the tile before, without branches, the scores' triangle is shared evenly by the waves, and the
// segments are one round of workgroups: a second would pay another fold and carry.
//   16384 x 80 x 128 x 64, q and k shared, prompts   333-352 us (fold 42, carry 11, walk 314, traced)
//   32768 x 16 x 128 x 128, prompts                  246-262 us (fold 79, carry 15, walk 180: 3.0 TB/s)
//   8192 x 16 x 128 x 128, gradients                 225-236 us (folds 43, carry 15, dq dk dv 176); in
//                                                    launches of their own, each a round of workgroups, 298
//   1001 x 6 x 64 x 50 fp32, gradients                50-54 us (folds 9, carry 8, dq dk dv 24, sums 11); apart 96
// Measured and no better: eight waves for 128 columns, swizzled rows instead of padded ones, rows without any bank
// conflict (half of them gone, the same time), three smaller workgroups per CU, scores dealt tile by tile to the
// waves, two heads per workgroup where they share q and k, nontemporal loads.
#include "linear_attention.h"

#include "seq_walk.h"
#include "vec.h"

namespace sss {

typedef __bf16 la_bf8 __attribute__((ext_vector_type(8)));
typedef float la_f4 __attribute__((ext_vector_type(4)));
typedef short la_s4 __attribute__((ext_vector_type(4)));
typedef uint32_t la_u4 __attribute__((ext_vector_type(4)));

// Eight values of a lane along a product's inner axis: lane l holds row (or column) l % 16 and
// inner indices 8 (l / 16) + 0..7 of 32.  fp32 products take eight steps of four inner indices, one
// element of each lane a step, so that both types have one layout.
template <bool BF16>
struct LaFrag;
template <>
struct LaFrag<true> {
  la_u4 u;
};
template <>
struct LaFrag<false> {
  float f[8];
};

__device__ __forceinline__ la_f4 la_mma(const LaFrag<true>& a, const LaFrag<true>& b, la_f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(la_bf8, a.u), __builtin_bit_cast(la_bf8, b.u), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ la_f4 la_mma(const LaFrag<false>& a, const LaFrag<false>& b, la_f4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.f[i], b.f[i], c, 0, 0, 0);
  return c;
}

// N parts that add up to v to 8 N bits: each the nearest bf16 to what the ones before leave.
// fp32: v itself.
template <int N>
__device__ __forceinline__ void la_split(const float (&v)[8], LaFrag<true> (&p)[N]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = vec_bf16_pair(rest[2 * i], rest[2 * i + 1]);
      p[n].u[i] = b;
      if (n + 1 < N) {
        rest[2 * i] -= __builtin_bit_cast(float, b << 16);
        rest[2 * i + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
      }
    }
  }
}
template <int N>
__device__ __forceinline__ void la_split(const float (&v)[8], LaFrag<false> (&p)[N]) {
  static_assert(N == 1, "fp32 takes one part");
#pragma unroll
  for (int i = 0; i < 8; ++i) p[0].f[i] = v[i];
}
__device__ __forceinline__ void la_widen(const LaFrag<true>& p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = p.u[i];
    v[2 * i] = __builtin_bit_cast(float, b << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, b & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void la_widen(const LaFrag<false>& p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p.f[i];
}

template <bool BF16>
__device__ __forceinline__ float la_get(const char* p) {
  if constexpr (BF16) return __builtin_bit_cast(float, (uint32_t)(*(const uint16_t*)p) << 16);
  else return *(const float*)p;
}

// LDS of one workgroup exchanged between its waves (global memory is not, within a launch)
__device__ __forceinline__ void la_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A tile in LDS: C rows of W elements, 16 bytes more between rows (so that 16 rows' pieces of 16
// bytes fall in different banks).
template <bool BF16, int W>
struct LaTile {
  static constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES, LD = W + VE;
  // inner axis along the row: row r0 + l % 16, columns c0 + 8 (l / 16) + 0..7
  static __device__ __forceinline__ LaFrag<BF16> rows(const char* t, int r0, int c0, int lane) {
    const char* const p = t + ((r0 + (lane & 15)) * LD + c0 + 8 * (lane >> 4)) * ES;
    LaFrag<BF16> f;
    if constexpr (BF16) {
      f.u = *(const la_u4*)p;
    } else {
      const la_f4 a = *(const la_f4*)p, b = *(const la_f4*)(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.f[i] = a[i], f.f[4 + i] = b[i];
    }
    return f;
  }
  // inner axis along the column: rows r0 + 8 (l / 16) + 0..7, for the lane's column: l % 16 = 4 a + b
  // stands for column c0 + A a + b.  bf16: the transposing read of LDS, in which the 16 lanes of a group
  // read four rows of 16 elements, lane i four of row i / 4, and lane l gets column l of them.
  template <int A>
  static __device__ __forceinline__ LaFrag<BF16> cols(const char* t, int r0, int c0, int lane) {
    const int l = lane & 15, g = lane >> 4;
    LaFrag<BF16> f;
    if constexpr (BF16) {
      typedef __attribute__((address_space(3))) la_s4* lds_p;
      const char* const p = t + ((r0 + 8 * g + (l >> 2)) * LD + c0 + A * (l & 3)) * ES;
      const la_s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)p);
      const la_s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p + 4 * LD * ES));
      const uint64_t lo = __builtin_bit_cast(uint64_t, a), hi = __builtin_bit_cast(uint64_t, b);
      f.u = la_u4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    } else {
      const char* const p = t + ((r0 + 8 * g) * LD + c0 + A * (l >> 2) + (l & 3)) * ES;
#pragma unroll
      for (int i = 0; i < 8; ++i) f.f[i] = *(const float*)(p + i * LD * ES);
    }
    return f;
  }
};

// A tile's scores in LDS: the 16 x 16 tiles on and below the diagonal (REV: above) and no others, bf16 as the sum of two
// parts.  A tile is pieces of 16 bytes of a row, the same piece of its 16 rows side by side, so that 16 lanes meet 256
// adjacent bytes.  (Rows as long as the tile, padded, took 9216 bytes for one part of 64 tokens: with two, a CU would
// hold one workgroup of the gradients in place of two.  This takes 10240 for both.)
template <bool BF16, int C, bool REV>
struct LaScores {
  static constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES, PARTS = BF16 ? 2 : 1, TI = C / 16, TILE = 256 * ES;
  static constexpr int PART = TI * (TI + 1) / 2 * TILE, kBytes = PARTS * PART;
  static __device__ __forceinline__ int tile(int it, int jt) {
    const int big = REV ? TI - 1 - it : it, small = REV ? TI - 1 - jt : jt;
    return (big * (big + 1) / 2 + small) * TILE;
  }
  // row l % 16 of row tile it, columns 32 ks + 8 (l / 16) + 0..7; the half of them that lies across the diagonal is zero
  static __device__ __forceinline__ LaFrag<BF16> rows(const char* part, int it, int ks, int lane) {
    const int l = lane & 15, g = lane >> 4;
    const bool half = REV ? 2 * ks < it : 2 * ks + 1 > it;  // one of the two tiles is not there
    const int only = REV ? 1 : 0;
    const int step = REV ? -TILE : TILE;  // to the next columns' tile
    const char* const p = part + tile(it, 2 * ks + (half ? only : 0)) + (half ? 0 : (g >> 1) * step) + (g & 1) * (8 / VE * 256) + l * 16;
    const bool in = !half || (g >> 1) == only;
    LaFrag<BF16> f;
    if constexpr (BF16) {
      f.u = *(const la_u4*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) f.u[i] = in ? f.u[i] : 0u;
    } else {
      const la_f4 a = *(const la_f4*)p, b = *(const la_f4*)(p + 256);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.f[i] = in ? a[i] : 0.0f, f.f[4 + i] = in ? b[i] : 0.0f;
    }
    return f;
  }
  // row l % 16, columns 4 (l / 16) + 0..3 of a tile
  static __device__ __forceinline__ void put(char* t, int it, int jt, int lane, const float (&v)[4]) {
    const int l = lane & 15, g = lane >> 4;
    char* const p = t + tile(it, jt) + l * 16;
    if constexpr (BF16) {
      typedef uint32_t u2 __attribute__((ext_vector_type(2)));
      const u2 hi = {vec_bf16_pair(v[0], v[1]), vec_bf16_pair(v[2], v[3])};
      const u2 lo = {vec_bf16_pair(v[0] - __builtin_bit_cast(float, hi[0] << 16), v[1] - __builtin_bit_cast(float, hi[0] & 0xFFFF0000u)),
                     vec_bf16_pair(v[2] - __builtin_bit_cast(float, hi[1] << 16), v[3] - __builtin_bit_cast(float, hi[1] & 0xFFFF0000u))};
      char* const q = p + (g >> 1) * 256 + 8 * (g & 1);
      *(u2*)q = hi;
      *(u2*)(q + PART) = lo;
    } else {
      *(la_f4*)(p + g * 256) = la_f4{v[0], v[1], v[2], v[3]};
    }
  }
  static __device__ __forceinline__ float get(const char* t, int i, int j) {
    const char* const p = t + tile(i >> 4, j >> 4) + ((j & 15) / VE) * 256 + (i & 15) * 16 + (j % VE) * ES;
    float v = la_get<BF16>(p);
    if constexpr (BF16) v += la_get<BF16>(p + PART);
    return v;
  }
};

// A tile on its way from memory to LDS, in registers of NT threads: pieces of 16 bytes, all loaded without a
// branch, so that they are in flight together.  Where a piece would lie outside the tile, the nearest one inside is
// loaded; what does not belong there is cleared when the tile is stored.
template <bool BF16, int C, int W, int NT>
struct LaLoad {
  using T = LaTile<BF16, W>;
  static constexpr int VE = T::VE, PER = W / VE, N = C * PER / NT;
  static_assert(N * NT == C * PER, "whole pieces");
  la_u4 v[N];
  static constexpr int RPT = NT / PER;  // rows at a time
  // rows first + r, r < nr, of `width` elements (strides are at most 2^24 elements: offsets in a tile fit 32 bits)
  __device__ __forceinline__ void load(int tid, const char* base, int64_t first, int64_t st, int nr, int width) {
    if (width < VE) return;  // store() does all
    const row_ptr p = row_at(base, first * st * T::ES);
    const uint32_t rb = (uint32_t)st * T::ES, c = (uint32_t)min(tid % PER * VE, width - VE) * T::ES;
    const uint32_t at = (uint32_t)(tid / PER) * rb + c, last = (uint32_t)(nr - 1) * rb + c;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const vec_u4 x = vec_get16<false>(p + min(at + (uint32_t)(n * RPT) * rb, last));
      v[n] = la_u4{x.x, x.y, x.z, x.w};
    }
  }
  // whether a value among those loaded is an infinity or no number (also one that the tile does not take)
  __device__ __forceinline__ bool wild() const {
    uint32_t any = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) any |= ((v[n][i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;  // an exponent of ones
        else any |= ((v[n][i] & 0x7F800000u) + 0x00800000u) & 0x80000000u;
      }
    return any != 0;
  }
  __device__ __forceinline__ void store(int tid, char* t, const char* base, int64_t first, int64_t st, int nr, int width) const {
    const int r0 = tid / PER, c = tid % PER * VE;
    char* const to = t + (r0 * T::LD + c) * T::ES;
    constexpr int step = RPT * T::LD * T::ES;
    if (nr == C && width == W) {
#pragma unroll
      for (int n = 0; n < N; ++n) *(la_u4*)(to + n * step) = v[n];
      return;
    }
    if (width < VE) {  // heads of a few elements: one by one
      for (int n = 0; n < N; ++n) {
        for (int i = 0; i < VE; ++i) {
          const bool in = r0 + n * RPT < nr && c + i < width;
          const char* const p = base + (first + min(r0 + n * RPT, nr - 1)) * st * T::ES + min(c + i, width - 1) * T::ES;
          if constexpr (BF16) ((uint16_t*)(to + n * step))[i] = in ? *(const uint16_t*)p : (uint16_t)0;
          else ((float*)(to + n * step))[i] = in ? *(const float*)p : 0.0f;
        }
      }
      return;
    }
    const int bits = c < width ? 8 * T::ES * max(c - (width - VE), 0) : 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      la_u4 x = v[n];
      if (width % VE != 0) {  // the row's last piece was loaded from before its place
        uint64_t lo = (uint64_t)x[1] << 32 | x[0], hi = (uint64_t)x[3] << 32 | x[2];
        if (bits >= 64) lo = hi >> (bits & 63), hi = 0;
        else if (bits > 0) lo = lo >> bits | hi << (64 - bits), hi >>= bits;
        x = la_u4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
      }
      const bool in = r0 + n * RPT < nr && c < width;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = in ? x[i] : 0u;
      *(la_u4*)(to + n * step) = x;
    }
  }
};

// Sums of a wave's lanes up to each lane, in the lanes' order.
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}
__device__ __forceinline__ double la_prefix(double v) {
  v += la_dpp<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8: within 16 lanes
  v += la_dpp<0x112, 0xF>(v);
  v += la_dpp<0x114, 0xF>(v);
  v += la_dpp<0x118, 0xF>(v);
  v += la_dpp<0x142, 0xA>(v);  // row_bcast 15: the sum of the 16 lanes before
  v += la_dpp<0x143, 0xC>(v);  // row_bcast 31: of the 32 before
  return v;
}
template <int CTRL>
__device__ __forceinline__ float la_dpp32(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ double la_lane(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// log decays up to kLaCut leave nothing of a state in fp32; kept finite, so that differences of
// their sums are numbers (a NaN stays one)
__device__ __forceinline__ double la_log2_decay(float g) { return (double)(g < kLaCut ? kLaCut : g) * 1.4426950408889634074; }

template <bool BF16, int E, int F, int MODE>
struct LaShape {
  static constexpr bool kRev = MODE == kLaFoldRev || MODE == kLaDk || MODE == kLaDv;
  static constexpr bool kOut = MODE >= kLaFwd;
  static constexpr bool kDots = MODE == kLaDq || MODE == kLaDk;
  static constexpr int XM = !BF16 ? 1 : kDots ? 3 : 2;          // parts of M as an operand
  static constexpr int UP = !BF16 ? 1 : MODE == kLaDv ? 2 : 3;  // of the weighted z
  static constexpr int NW = F == 256 ? 8 : 4, NT = NW * 64, NF = F / (16 * NW);
  static constexpr int C = BF16 ? kLaTile : kLaTile / 2, TI = C / 16, KS = C / 32;
  static constexpr int NS = TI * (TI + 1) / 2, SPW = (NS + NW - 1) / NW;  // tiles of scores that are not zero; per wave
  // LDS: the tiles x, y, z, w and scores, weights of y z^T, beta, sums of the columns' waves, two flags
  static constexpr int ROWX = LaTile<BF16, E>::LD * (BF16 ? 2 : 4) * C, ROWZ = LaTile<BF16, F>::LD * (BF16 ? 2 : 4) * C;
  static constexpr int kY = kOut ? ROWX : 0, kZ = kY + ROWX, kW = kZ + ROWZ, kP = kW + (kDots ? ROWZ : 0);
  static constexpr int kU = kP + (kOut ? LaScores<BF16, C, kRev>::kBytes : 0), kB = kU + 4 * C, kR = kB + 4 * C;
  static constexpr int kWild = kR + (kDots ? 4 * NW * C : 0), kBytes = kWild + 16;
};

// One segment and head; id: of the workgroup among those of the walk.
template <bool BF16, int E, int F, int MODE>
__device__ __forceinline__ void la_walk(const LaWalk& g, char* smem, unsigned id) {
  using S = LaShape<BF16, E, F, MODE>;
  constexpr int NW = S::NW, NT = S::NT, NF = S::NF, C = S::C, TI = S::TI, KS = S::KS, ET = E / 16, EK = E / 32;
  constexpr bool kRev = S::kRev, kOut = S::kOut, kDots = S::kDots;
  constexpr int ES = BF16 ? 2 : 4;
  using TX = LaTile<BF16, E>;
  using TZ = LaTile<BF16, F>;
  using TP = LaScores<BF16, C, kRev>;
  char* const lx = smem;
  char* const ly = smem + S::kY;
  char* const lz = smem + S::kZ;
  char* const lw = smem + S::kW;
  char* const lp = smem + S::kP;
  float* const luw = (float*)(smem + S::kU);    // weights of y z^T
  float* const lbeta = (float*)(smem + S::kB);  // beta
  float* const lrr = (float*)(smem + S::kR);    // sums over the columns of each wave
  int* const lwild = (int*)(smem + S::kWild);   // a tile's z has a value that is not finite (alternating tiles)
  // between the rows of z: the sums of log2 decays; of y: the weights of x M, and the waves' parts of a
  // sum
  auto lg = [&](int i) __attribute__((always_inline)) { return (double*)(lz + (i * TZ::LD + F) * ES); };
  auto lsr = [&](int i) __attribute__((always_inline)) { return (float*)(ly + (i * TX::LD + E) * ES); };
  auto lred = [&](int i) __attribute__((always_inline)) { return (float*)(ly + (i * TX::LD + E) * ES + 4); };

  auto uni = [](int v) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(v); };
  const int lane = threadIdx.x & 63;
  const int wave_id = uni((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, l4 = lane >> 4;
  const int h = uni((int)(id % (unsigned)g.H));
  int seg = uni((int)(id / (unsigned)g.H));
  if constexpr (MODE == kLaFoldRev) ++seg;  // the first segment has no edge on its left
  const int c0 = seg * g.K, tend = min(c0 + g.K, g.tokens);
  const LaBounds cu(g.cu, g.nseq, lane);
  // slots and starts of the first 64 sequences, with the boundaries
  int my_slot = lane, my_init = 0;
  if (g.state != nullptr && g.nseq > 0) {
    if (g.sidx != nullptr) my_slot = g.sidx[min(lane, g.nseq - 1)];
    if (g.init != nullptr) my_init = g.init[min(lane, g.nseq - 1)];
  }
  const int lo = min(max(cu.at(0), 0), g.tokens), hi = min(max(cu.at(g.nseq), 0), g.tokens);
  const int f0 = wave_id * (16 * NF);  // the wave's columns
  const int Ew = g.y.width, Fw = g.z.width;
  const char* const xp = kOut ? g.x.p + uni(h / g.x.rep) * g.x.sh * ES : nullptr;
  const char* const yp = g.y.p + uni(h / g.y.rep) * g.y.sh * ES;
  const char* const zp = g.z.p + uni(h / g.z.rep) * g.z.sh * ES;
  const char* const wp = kDots ? g.w.p + uni(h / g.w.rep) * g.w.sh * ES : nullptr;

  const float* const gp = g.g + h;
  const float* const bp = g.beta != nullptr ? g.beta + h : nullptr;
  const float skip = (MODE == kLaFwd || MODE == kLaDv) && g.D != nullptr ? g.D[h] : 0.0f;

  la_f4 M[ET][NF];
  // Element r of a lane's accumulator t is row 32 (t / 2) + 8 (l / 16) + 4 (t % 2) + r of M.  fn(value, offset
  // in a head's state) for those inside the head's sizes.  The offsets start from values that the compiler
  // does not know, or it keeps all of them, for every accumulator, in registers over the loops.
  auto each = [&](auto&& fn) __attribute__((always_inline)) {
    int e0 = 8 * l4, f1 = f0 + l16;
    asm volatile("" : "+v"(e0), "+v"(f1));
    const int se = (int)g.se, sf = (int)g.sf;
    const int at = e0 * se + f1 * sf;
#pragma unroll
    for (int t = 0; t < ET; ++t)
#pragma unroll
      for (int nf = 0; nf < NF; ++nf)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int e = 32 * (t >> 1) + 4 * (t & 1) + r;
          if (e0 < Ew - e && f1 < Fw - 16 * nf) {
            float v = M[t][nf][r];
            fn(v, at + e * se + 16 * nf * sf);
            M[t][nf][r] = v;
          }
        }
  };
  auto zero = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < ET; ++t)
#pragma unroll
      for (int nf = 0; nf < NF; ++nf) M[t][nf] = la_f4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // all loads in flight together: what lies outside the head's sizes is loaded from inside and cleared
  auto peek = [&](const float* p, auto&& fn) __attribute__((always_inline)) {
    int e0 = 8 * l4, f1 = f0 + l16;
    asm volatile("" : "+v"(e0), "+v"(f1));
    const int se = (int)g.se, sf = (int)g.sf;
    la_f4 v[ET][NF];
    if (kDots && Ew % 4 == 0) {  // se is 1: four rows are 16 adjacent bytes
#pragma unroll
      for (int t = 0; t < ET; ++t)
#pragma unroll
        for (int nf = 0; nf < NF; ++nf) {
          const vec_u4 x = *(const vec_u4*)(p + (min(e0 + 32 * (t >> 1) + 4 * (t & 1), Ew - 4) + min(f1 + 16 * nf, Fw - 1) * sf));
          v[t][nf] = __builtin_bit_cast(la_f4, x);
        }
    } else {
#pragma unroll
      for (int t = 0; t < ET; ++t)
#pragma unroll
        for (int nf = 0; nf < NF; ++nf)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[t][nf][r] = p[min(e0 + 32 * (t >> 1) + 4 * (t & 1) + r, Ew - 1) * se + min(f1 + 16 * nf, Fw - 1) * sf];
    }
#pragma unroll
    for (int t = 0; t < ET; ++t)
#pragma unroll
      for (int nf = 0; nf < NF; ++nf)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool in = e0 < Ew - (32 * (t >> 1) + 4 * (t & 1) + r) && f1 < Fw - 16 * nf;
          M[t][nf][r] = fn(M[t][nf][r], in ? v[t][nf][r] : 0.0f);
        }
  };
  auto from = [&](const float* p) __attribute__((always_inline)) {  // null: zero
    if (p == nullptr) zero();
    else peek(p, [](float, float v) __attribute__((always_inline)) { return v; });
  };
  auto to = [&](float* p) __attribute__((always_inline)) {
    each([&](float& v, int o) __attribute__((always_inline)) { p[o] = v; });
  };
  const int64_t per = g.hs, at_seg = ((int64_t)seg * g.H + h) * per;
  auto of_seq = [&](int64_t s) __attribute__((always_inline)) { return (s * g.H + h) * per; };

  if (threadIdx.x == 0) lwild[0] = lwild[1] = 0;
  int turn = 0;

  double total = 0.0;  // log2 of the decay over a folded part
  float trace = 0.0f, through = 0.0f;

  // tokens a .. e-1, of one sequence; adj: the adjoint behind them (null: zero), for `through`
  auto walk = [&](int a, int e, const float* adj) __attribute__((always_inline)) {
    LaLoad<BF16, C, E, NT> rx, ry;
    LaLoad<BF16, C, F, NT> rz, rw;
    float rg = 0.0f, rb = 0.0f;
    const int ntile = (e - a + C - 1) / C;
    // Parts: 1, the decays and x; 2, y; 4, z and w.  Asked for at three points of the tile before, so that none of them
    // waits for room among the loads in flight: at one point, 349 us in place of 343 for prompts of 16384 x 80 x 128 x 64,
    // 248 in place of 239 for the gradients of 8192 x 16 x 128 x 128.
    auto fetch = [&](int tid, int m, int part) __attribute__((always_inline)) {
      const int lane = tid & 63;
      const int t = a + m * C, nr = min(C, e - t);
      // first, so that waiting for them does not wait for the tiles: vector loads return in order
      const int r = t + min(lane, nr - 1);
      if (part & 1) {
        rg = gp[r * g.g_st];
        rb = bp != nullptr ? bp[r * g.beta_st] : 1.0f;
      }
      if (kOut && (part & 1)) rx.load(tid, xp, t, g.x.st, nr, Ew);
      if (part & 2) ry.load(tid, yp, t, g.y.st, nr, Ew);
      if (part & 4) rz.load(tid, zp, t, g.z.st, nr, Fw);
      if (kDots && (part & 4)) rw.load(tid, wp, t, g.w.st, nr, Fw);
    };
    fetch((int)threadIdx.x, kRev ? ntile - 1 : 0, 7);
    for (int k = 0; k < ntile; ++k) {
      const int m = kRev ? ntile - 1 - k : k;
      const int t0 = a + m * C, nr = min(C, e - t0);
      // addresses in a tile start from values that the compiler does not know, or it keeps them all in registers
      // over the loop, and these are short
      int tid = (int)threadIdx.x, wave = wave_id;
      asm volatile("" : "+v"(tid), "+s"(wave));
      const int lane = tid & 63, l16 = tid & 15, l4 = lane >> 4, f0 = wave * (16 * NF);
      if constexpr (MODE == kLaFwd) __builtin_amdgcn_s_setprio(0);
      la_barrier();  // the tile before has been read
      const bool alive = lane < nr;
      const double x = la_prefix(la_log2_decay(alive ? rg : 0.0f)), tot = la_lane(x, 63);
      const float b = alive ? rb : 0.0f, keep = fast_exp2((float)tot);
      if constexpr (!kOut) total += tot;
      // the tokens that nothing before them reaches
      const uint64_t cuts = MODE == kLaDq ? __builtin_amdgcn_ballot_w64(alive && rg <= kLaCut) : 0;
      if (wave == 0 && lane < C) {
        const float in = fast_exp2((float)x), out = fast_exp2((float)(tot - x));
        *lg(lane) = x;
        *lsr(lane) = kRev ? out : g.scale * in;
        luw[lane] = kRev ? g.scale * in : b * out;
        lbeta[lane] = b;
      }
      if constexpr (kOut) rx.store(tid, lx, xp, t0, g.x.st, nr, Ew);
      ry.store(tid, ly, yp, t0, g.y.st, nr, Ew);
      rz.store(tid, lz, zp, t0, g.z.st, nr, Fw);
      if constexpr (kOut) {
        turn ^= 1;
        if (Fw < TZ::VE || rz.wild()) lwild[turn] = 1;
      }
      if constexpr (kDots) rw.store(tid, lw, wp, t0, g.w.st, nr, Fw);
      la_barrier();
      if (k + 1 < ntile) fetch(tid, kRev ? m - 1 : m + 1, kOut ? 1 : 7);
      if constexpr (MODE == kLaDq) {
        if (k + 1 == ntile) {
          through = 0.0f;
          if (adj != nullptr) {
            peek(adj, [&](float m, float v) __attribute__((always_inline)) {
              through = __builtin_fmaf(m, v, through);
              return m;
            });
            through *= keep;
          }
        }
      }

      LaFrag<BF16> zf[KS][NF];  // z by columns
      auto take_z = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int nf = 0; nf < NF; ++nf) zf[ks][nf] = TZ::template cols<4>(lz, 32 * ks, f0 + 16 * nf, lane);
      };
      if constexpr (kOut) {
        // Scores, transposed: the lane has row i, columns j + r.  The waves share the 16 x 16 tiles on and below
        // (backwards: above) the diagonal.
#pragma unroll
        for (int q = 0; q < S::SPW; ++q) {
          const int n = wave + q * NW;
          if (n >= S::NS) break;
          const int big = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, small = n - big * (big + 1) / 2;
          const int it = kRev ? TI - 1 - big : big, jt = kRev ? TI - 1 - small : small;
          const int i = 16 * it + l16, j = 16 * jt + 4 * l4;
          la_f4 sc = {0.0f, 0.0f, 0.0f, 0.0f}, other = sc;
#pragma unroll
          for (int s = 0; s < EK; ++s) sc = la_mma(TX::rows(ly, 16 * jt, 32 * s, lane), TX::rows(lx, 16 * it, 32 * s, lane), sc);
          if constexpr (MODE == kLaDq) {  // q k^T
#pragma unroll
            for (int s = 0; s < F / 32; ++s)
              other = la_mma(TZ::rows(lz, 16 * jt, 32 * s, lane), TZ::rows(lw, 16 * it, 32 * s, lane), other);
          }
          const double gi = *lg(i);
          const float row_w = kRev ? lbeta[i] * g.scale : g.scale;
          const la_f4 bj = *(const la_f4*)(lbeta + j);
          float p[4], ci[4], ri = 0.0f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const double d = kRev ? *lg(j + r) - gi : gi - *lg(j + r);
            const bool in = kRev ? j + r >= i : j + r <= i;
            const float wt = row_w * fast_exp2((float)d), b = kRev ? 1.0f : bj[r];
            p[r] = in ? wt * b * sc[r] : 0.0f;
            if constexpr (MODE == kLaDq) {
              ci[r] = in ? wt * sc[r] * other[r] : 0.0f;
              ri += b * ci[r];
              trace += j + r == i ? sc[r] : 0.0f;
            }
            if constexpr (MODE == kLaFwd || MODE == kLaDv) p[r] += j + r == i ? skip : 0.0f;
          }
          TP::put(lp, it, jt, lane, p);
          if constexpr (MODE == kLaDq) {  // sums over the tile's columns and rows, kept between the rows of x and of w
            ri += __shfl_xor(ri, 16);
            ri += __shfl_xor(ri, 32);
            if (l4 == 0) *(float*)(lx + (i * TX::LD + E) * ES + 4 * jt) = ri;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float v = ci[r];
              v += la_dpp32<0xB1>(v);   // quad_perm [1,0,3,2]
              v += la_dpp32<0x4E>(v);   // quad_perm [2,3,0,1]
              v += la_dpp32<0x141>(v);  // row_half_mirror
              v += la_dpp32<0x140>(v);  // row_mirror
              if (l16 == 0) *(float*)(lw + ((j + r) * TZ::LD + F) * ES + 4 * it) = v;
            }
          }
        }
        if (k + 1 < ntile) fetch(tid, kRev ? m - 1 : m + 1, 2);
        // The outputs' products before what the CU's other workgroup does between them (16384 x 80 x 128 x 64 339 -> 332 us;
        // the gradients, whose three walks share the GPU, were 3% slower with it).
        if constexpr (MODE == kLaFwd) __builtin_amdgcn_s_setprio(1);
        // x M, transposed: the lane has row i of the tokens, columns f + r
        la_f4 o[TI][NF];
#pragma unroll
        for (int t = 0; t < TI; ++t)
#pragma unroll
          for (int nf = 0; nf < NF; ++nf) o[t][nf] = la_f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < EK; ++s) {
          LaFrag<BF16> mf[NF][S::XM];
#pragma unroll
          for (int nf = 0; nf < NF; ++nf) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = M[2 * s][nf][r], v[4 + r] = M[2 * s + 1][nf][r];
            la_split<S::XM>(v, mf[nf]);
          }
          LaFrag<BF16> xf[TI];
#pragma unroll
          for (int t = 0; t < TI; ++t) xf[t] = TX::rows(lx, 16 * t, 32 * s, lane);
#pragma unroll
          for (int q = S::XM - 1; q >= 0; --q)
#pragma unroll
            for (int t = 0; t < TI; ++t)
#pragma unroll
              for (int nf = 0; nf < NF; ++nf) o[t][nf] = la_mma(mf[nf][q], xf[t], o[t][nf]);
        }
#pragma unroll
        for (int t = 0; t < TI; ++t) {
          const float sr = *lsr(16 * t + l16), rb_ = kRev ? lbeta[16 * t + l16] : 1.0f;
          float dot = 0.0f;
#pragma unroll
          for (int nf = 0; nf < NF; ++nf) {
            o[t][nf] *= sr;
            if constexpr (kDots) {
              const char* const pw = lw + ((16 * t + l16) * TZ::LD + f0 + 16 * nf + 4 * l4) * ES;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                dot = __builtin_fmaf(la_get<BF16>(pw + ES * r), o[t][nf][r], dot);
              }
            }
            if constexpr (kRev) o[t][nf] *= rb_;
          }
          if constexpr (kDots) {
            dot += __shfl_xor(dot, 16);
            dot += __shfl_xor(dot, 32);
            if (l4 == 0) lrr[wave * C + 16 * t + l16] = dot;
          }
        }
        if (k + 1 < ntile) fetch(tid, kRev ? m - 1 : m + 1, 4);
        take_z();
        if (threadIdx.x == 0) lwild[turn ^ 1] = 0;  // last read before this tile
        la_barrier();  // the scores are there
        const bool wild = uni(lwild[turn]) != 0;
        if constexpr (kDots) {
          if (wave == 0) {  // C tokens, a lane each
            const int i2 = lane & (C - 1);
            const bool in = lane < nr;
            const int64_t at = (int64_t)h * g.tokens + t0 + i2;
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < NW; ++q) v += lrr[q * C + i2];
            if (in) (MODE == kLaDq ? g.rows : g.cols2)[at] = v;
            if constexpr (MODE == kLaDq) {
              float rs = 0.0f, cs = 0.0f;
#pragma unroll
              for (int q = 0; q < TI; ++q) {
                rs += q <= i2 / 16 ? *(const float*)(lx + (i2 * TX::LD + E) * ES + 4 * q) : 0.0f;
                cs += q >= i2 / 16 ? *(const float*)(lw + (i2 * TZ::LD + F) * ES + 4 * q) : 0.0f;
              }
              // Summed from the right.  Tokens behind a cut add up to zero, but in their roundings alone, which would reach the
              // tokens before it: none is taken from lanes that have one between.
              float n = lane < C ? rs - lbeta[i2] * cs : 0.0f;
              const uint64_t behind = cuts >> lane >> 1;
#pragma unroll
              for (int d = 1; d < C; d *= 2) {
                const float up = __shfl_down(n, d);
                if (lane + d < C && (behind & (((uint64_t)1 << d) - 1)) == 0) n += up;
              }
              if (in) {
                g.within[at] = n;
                g.cols[at] = cs;
              }
            }
          }
        }
        const bool wide = !BF16 || (kDots && g.out_f32);
        const uint32_t out_es = wide ? 4 : 2, out_row = (uint32_t)g.out_st * out_es;
        const row_ptr to_out = row_at(g.out, ((int64_t)t0 * g.out_st + h * g.out_sh) * out_es);
        if (!wild) {
          // the rows' products in turn, so that none waits for the one before (16384 x 80 x 128 x 64: 373 us row by row, 361 in
          // turn, 353 with those of x M in turn as well)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int q = TP::PARTS - 1; q >= 0; --q)
#pragma unroll
              for (int t = 0; t < TI; ++t) {
                if (kRev ? 2 * ks + 1 < t : 2 * ks > t) continue;
                const LaFrag<BF16> pf = TP::rows(lp + q * TP::PART, t, ks, lane);
#pragma unroll
                for (int nf = 0; nf < NF; ++nf) o[t][nf] = la_mma(zf[ks][nf], pf, o[t][nf]);
              }
        } else {
          // a score of zero times an infinity or no number of a token that this row does not see would be no number:
          // the products that count, one by one
#pragma unroll
          for (int t = 0; t < TI; ++t) {
            const int i2 = 16 * t + l16;
#pragma unroll 1
            for (int j = 0; j < C; ++j) {
              if (kRev ? j < i2 : j > i2) continue;
              const float p = TP::get(lp, i2, j);
#pragma unroll
              for (int nf = 0; nf < NF; ++nf)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  o[t][nf][r] = __builtin_fmaf(p, la_get<BF16>(lz + (j * TZ::LD + f0 + 16 * nf + 4 * l4 + r) * ES), o[t][nf][r]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < TI; ++t) {
          const int i2 = 16 * t + l16;
          if (i2 >= nr) continue;
#pragma unroll
          for (int nf = 0; nf < NF; ++nf) {
            const int f = f0 + 16 * nf + 4 * l4;
            const uint32_t at = (uint32_t)i2 * out_row + (uint32_t)f * out_es;
            const float v[4] = {o[t][nf][0], o[t][nf][1], o[t][nf][2], o[t][nf][3]};
            if (BF16 && !wide) {
              Vec<true, 4> r;
              r.set(v);
              if (Fw == F || f + 4 <= Fw) r.store(to_out, at);
              else r.store_first(to_out, at, Fw - f);
            } else {
              Vec<false, 4> r;
              r.set(v);
              if (Fw == F || f + 4 <= Fw) r.store(to_out, at);
              else r.store_first(to_out, at, Fw - f);
            }
          }
        }
      }

      if constexpr (!kOut) take_z();
      // M <- e^(G_C) M + sum_j weight_j y_j z_j^T; of the parts of a product none waits for the one before, as above
      // (16384 x 80 x 128 x 64 315 -> 307 us, gradients of 8192 x 16 x 128 x 128 216 -> 211)
#pragma unroll
      for (int t = 0; t < ET; ++t)
#pragma unroll
        for (int nf = 0; nf < NF; ++nf) M[t][nf] *= keep;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        LaFrag<BF16> wz[NF][S::UP];
        const la_f4 u0 = *(const la_f4*)(luw + 32 * ks + 8 * l4), u1 = *(const la_f4*)(luw + 32 * ks + 8 * l4 + 4);
#pragma unroll
        for (int nf = 0; nf < NF; ++nf) {
          float v[8];
          la_widen(zf[ks][nf], v);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] *= u0[r], v[4 + r] *= u1[r];
          la_split<S::UP>(v, wz[nf]);
        }
#pragma unroll
        for (int t = 0; t < ET; t += 4) {
          LaFrag<BF16> yf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) yf[i] = TX::template cols<8>(ly, 32 * ks, 32 * ((t + i) >> 1) + 4 * ((t + i) & 1), lane);
#pragma unroll
          for (int q = S::UP - 1; q >= 0; --q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int nf = 0; nf < NF; ++nf) M[t + i][nf] = la_mma(yf[i], wz[nf][q], M[t + i][nf]);
        }
      }
    }
  };

  // the same value in every thread
  auto block_sum = [&](float v) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    la_barrier();
    if (lane == 0) *lred(wave_id) = v;
    la_barrier();
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < NW; ++q) s += *lred(q);
    return s;
  };

  auto slot_of = [&](int s) __attribute__((always_inline)) {  // -1: none
    if (g.state == nullptr) return -1;
    const int slot = g.nseq <= 64 ? __builtin_amdgcn_readlane(my_slot, s) : g.sidx != nullptr ? uni(g.sidx[s]) : s;
    return (unsigned)slot < (unsigned)g.slots ? slot : -1;
  };
  auto continues = [&](int s) __attribute__((always_inline)) {  // its slot's state
    if (g.state == nullptr || g.init == nullptr) return false;
    return (g.nseq <= 64 ? __builtin_amdgcn_readlane(my_init, s) : uni(g.init[s])) != 0;
  };

  if constexpr (!kOut) {
    // the sequence that runs across this segment's right (left) edge
    int flag = 0;  // 0: none; 1: it runs across the other edge too; 2: it begins (ends) in the segment
    const int edge = kRev ? c0 : tend;
    if (edge > lo && edge < hi) {
      const int s = cu.find(kRev ? c0 : tend - 1);
      const int end = min(cu.at(s + 1), hi), beg = max(cu.at(s), 0);
      if (kRev ? beg < c0 && end > c0 : beg < tend && end > tend) {
        flag = (kRev ? end <= tend : beg >= c0) ? 2 : 1;
        const float* src = nullptr;
        if (flag == 2) {
          if (g.from != nullptr) src = g.from + of_seq(s);
          else if (slot_of(s) >= 0 && continues(s)) src = g.state + of_seq(slot_of(s));
        }
        from(src);
        // for the second pass: the slot itself is overwritten there, by another workgroup
        if (src != nullptr && g.begin != nullptr) to(g.begin + at_seg);
        walk(kRev ? c0 : max(beg, c0), kRev ? min(end, tend) : tend, nullptr);
        to(g.end + at_seg);
        if (threadIdx.x == 0) g.sum[(int64_t)seg * g.H + h] = (float)total;
      }
    }
    if (h == 0 && threadIdx.x == 0) g.flag[seg] = flag;
  } else {
    int t = max(c0, lo);
    const int stop = min(tend, hi);
    if constexpr (MODE != kLaFwd) {  // gradients of tokens outside every sequence are zero
      const int gap0 = min(t, tend), gap1 = max(stop, c0);
      auto clear = [&](int a, int b) __attribute__((always_inline)) {
        const int n = (b - a) * Fw;
        for (int i = threadIdx.x; i < n; i += NT) {
          const int64_t at = (int64_t)(a + i / Fw) * g.out_st + h * g.out_sh + i % Fw;
          if (BF16 && !g.out_f32) ((uint16_t*)g.out)[at] = 0;
          else ((float*)g.out)[at] = 0.0f;
        }
      };
      clear(c0, gap0);
      clear(max(gap1, gap0), tend);
    }
    int s = t < stop ? cu.find(t) : 0;
    while (t < stop) {
      const int end = min(cu.at(s + 1), hi);
      if (end <= t) {  // past this sequence (or an empty one)
        if (++s >= g.nseq) break;
        continue;
      }
      const int e = min(end, tend);
      const bool before = began_before(cu.at(s), c0), after = end > tend;
      if constexpr (MODE == kLaFwd) {
        const int slot = slot_of(s);
        const bool old = slot >= 0 && continues(s);
        from(before ? g.enter + at_seg : !old ? nullptr : after ? g.begin + at_seg : g.state + of_seq(slot));
        walk(t, e, nullptr);
        if (!after && slot >= 0) to(g.state + of_seq(slot));
      } else if constexpr (MODE == kLaDq) {
        from(before ? g.enter + at_seg : g.from != nullptr ? g.from + of_seq(s) : nullptr);
        const float* const adj = after ? g.back + at_seg : g.dfinal != nullptr ? g.dfinal + of_seq(s) : nullptr;
        walk(t, e, adj);
        const float v = adj != nullptr ? block_sum(through) : 0.0f;
        if (threadIdx.x == 0) (after ? g.edge[(int64_t)seg * g.H + h] : g.last[(int64_t)s * g.H + h]) = v;
      } else {
        from(after ? g.enter + at_seg : g.from != nullptr ? g.from + of_seq(s) : nullptr);
        walk(t, e, nullptr);
        if (MODE == kLaDk && !before && g.to != nullptr) to(g.to + of_seq(s));
      }
      t = e;
    }
    if constexpr (MODE == kLaDq) {
      if (g.trace != nullptr) {
        const float v = block_sum(trace);
        if (threadIdx.x == 0) g.trace[(int64_t)seg * g.H + h] = v;
      }
    }
  }
}

template <int E, int F>
constexpr int kLaThreads = F == 256 ? 512 : 256;
template <int E, int F>
constexpr int kLaWaves = E == 256 && F < 256 ? 1 : 2;  // per SIMD, at least

template <bool BF16, int E, int F, int MODE>
__global__ __launch_bounds__((kLaThreads<E, F>), (kLaWaves<E, F>)) void la_walk_kernel(LaWalk g) {
  __shared__ __attribute__((aligned(16))) char smem[LaShape<BF16, E, F, MODE>::kBytes];
  la_walk<BF16, E, F, MODE>(g, smem, xcd_remap(blockIdx.x, gridDim.x));
}

// The gradients' walks in one launch each for what does not wait for each other: both folds, and dq with dk, and dv where
// its state has the same sizes.  n: workgroups of each.
constexpr int la_most(int a, int b) { return a > b ? a : b; }

template <bool BF16, int E, int F>
__global__ __launch_bounds__((kLaThreads<E, F>), (kLaWaves<E, F>)) void la_folds_kernel(LaWalk fwd, LaWalk rev, unsigned n) {
  __shared__ __attribute__((aligned(16)))
  char smem[la_most(LaShape<BF16, E, F, kLaFoldFwd>::kBytes, LaShape<BF16, E, F, kLaFoldRev>::kBytes)];
  if (blockIdx.x < n) la_walk<BF16, E, F, kLaFoldFwd>(fwd, smem, xcd_remap(blockIdx.x, n));
  else la_walk<BF16, E, F, kLaFoldRev>(rev, smem, xcd_remap(blockIdx.x - n, n));
}

template <bool BF16, int E, int F>
__global__ __launch_bounds__((kLaThreads<E, F>), (kLaWaves<E, F>)) void la_grads_kernel(LaWalk dq, LaWalk dk, LaWalk dv, unsigned n) {
  __shared__ __attribute__((aligned(16)))
  char smem[la_most(LaShape<BF16, E, F, kLaDq>::kBytes, LaShape<BF16, E, F, kLaDk>::kBytes)];
  static_assert(LaShape<BF16, E, F, kLaDv>::kBytes <= sizeof(smem), "dv's tiles are fewer");
  if (blockIdx.x < n) la_walk<BF16, E, F, kLaDq>(dq, smem, xcd_remap(blockIdx.x, n));
  else if (blockIdx.x < 2 * n) la_walk<BF16, E, F, kLaDk>(dk, smem, xcd_remap(blockIdx.x - n, n));
  else if constexpr (E == F) la_walk<BF16, E, F, kLaDv>(dv, smem, xcd_remap(blockIdx.x - 2 * n, n));
}

#ifdef SSS_INST_E
template <int E, int F>
hipError_t la_run(LaMode mode, bool bf16, const LaWalk& g, unsigned grid, hipStream_t stream) {
  const dim3 block(kLaThreads<E, F>);
#define SSS_LA_MODE(MODE)                                                                                          \
  if (mode == MODE) {                                                                                              \
    if (bf16) hipLaunchKernelGGL((la_walk_kernel<true, E, F, MODE>), dim3(grid), block, 0, stream, g);             \
    else hipLaunchKernelGGL((la_walk_kernel<false, E, F, MODE>), dim3(grid), block, 0, stream, g);                 \
    return hipGetLastError();                                                                                      \
  }
  SSS_LA_MODE(kLaFoldFwd)
  SSS_LA_MODE(kLaFwd)
  if constexpr (E != F) {
    SSS_LA_MODE(kLaDv)
  }
#undef SSS_LA_MODE
  return hipErrorInvalidValue;
}

template <int E, int F>
hipError_t la_run_folds(bool bf16, const LaWalk& fwd, const LaWalk& rev, unsigned n, hipStream_t stream) {
  const dim3 block(kLaThreads<E, F>);
  if (bf16) hipLaunchKernelGGL((la_folds_kernel<true, E, F>), dim3(2 * n), block, 0, stream, fwd, rev, n);
  else hipLaunchKernelGGL((la_folds_kernel<false, E, F>), dim3(2 * n), block, 0, stream, fwd, rev, n);
  return hipGetLastError();
}

template <int E, int F>
hipError_t la_run_grads(bool bf16, const LaWalk& dq, const LaWalk& dk, const LaWalk& dv, unsigned n, hipStream_t stream) {
  const dim3 block(kLaThreads<E, F>), grid((E == F ? 3 : 2) * n);
  if (bf16) hipLaunchKernelGGL((la_grads_kernel<true, E, F>), grid, block, 0, stream, dq, dk, dv, n);
  else hipLaunchKernelGGL((la_grads_kernel<false, E, F>), grid, block, 0, stream, dq, dk, dv, n);
  return hipGetLastError();
}

template hipError_t la_run<SSS_INST_E, SSS_INST_F>(LaMode, bool, const LaWalk&, unsigned, hipStream_t);
template hipError_t la_run_folds<SSS_INST_E, SSS_INST_F>(bool, const LaWalk&, const LaWalk&, unsigned, hipStream_t);
template hipError_t la_run_grads<SSS_INST_E, SSS_INST_F>(bool, const LaWalk&, const LaWalk&, const LaWalk&, unsigned, hipStream_t);
#endif

}  // namespace sss

// packed_scan.hip -- gfx950 kernels of the selective scan over packed prompts, with the state
// of every sequence in a cache slot.
//
// Per sequence, channel d and state n, with the step size dt = delta, or delta + bias, or
// softplus of that:
//   h_t = exp(dt_t A[d,n]) h_{t-1} + dt_t B_t[n] x_t,  y_t = (sum_n C_t[n] h_t[n] + D[d] x_t) silu(z_t)
// from the slot's state (or zero), which the sequence's last state replaces.
//
// The mapping of a step is that of selective_scan.hip: one wave = 64 adjacent channels, each
// lane walks time with its states in registers, B/C rows are staged in LDS and read by broadcast.  The
// packed axis is cut into chunks of K tokens without regard to the sequences, whose lengths
// only the device knows: the launch needs the token count alone.  At most one sequence runs
// across the end of a chunk, so that
//   pass 1 folds, in each chunk, only the tokens of the sequence that goes on into the next
//          one: from zero (with the sum of its step sizes) where it began earlier, from its
//          initial state where it begins in this chunk;
//   carry  composes these along each sequence, h = exp(A sum dt) h + h_chunk, into the state
//          entering each chunk;
//   pass 2 walks every chunk's sequences, writes y, and the final states to the slots.
// Short sequences thus cost no second pass over their tokens: with lengths well below K nearly
// nothing runs in pass 1.  (9001 tokens x 2048 in 40 sequences has K = 71: 82-87% of the tokens lie in
// one that goes on, and are walked twice.)
//
// Bound by the issue of VALU instructions: 32768 x 5120 x 16 in three sequences takes 388 us (pass
// 1) + 21 (carry) + 528 (pass 2) on a traced run, 858-902 untraced.  Per wave and step pass 1 issues 17
// exps, two slots of four clocks each, and 65 other instructions, pass 2 19 and 90: 421 and 549 us at
// 2.4 GHz if no two waves' instructions issue together, 292 and 367 if all but the exps do.  The memory
// traffic, 706 and 1450 MB, would take 133 and 274; 58 MB of the latter are 28 registers per lane that
// pass 2, at its limit of 128, keeps in scratch memory over the loop over sequences.
//
// A slot is read in pass 1 (or in pass 2 by the wave that also writes it), so that it is updated in
// place.
#include "front.h"
#include "seq_walk.h"
#include "vec.h"
#include "kernels.h"

#include <algorithm>

namespace sss {

struct PScanGeo {
  int64_t sx, sd, sz, sb, sc;  // elements between tokens of x, delta, z, B, C
  int tokens, nseq, slots, D, K, ngroups, gpb, nblk;
  int piece;  // tokens whose rows stay within 32-bit byte offsets of the first
  int bc_bf16;
};

constexpr int pscan_min_waves(int ns) { return ns >= 64 ? 1 : ns >= 32 ? 2 : 4; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t pscan_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7FFFFFFF, 0x00020000);
}
__device__ __forceinline__ float pscan_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t pscan_u32(float f) { return __builtin_bit_cast(uint32_t, f); }

// softplus(v) = max(v, 0) + log1p(e), e = e^-|v|, with log1p(e) = e p(e) on [0, 1]: p is the polynomial of
// degree 8 with the least relative error there (fitted by linear programming on Chebyshev nodes;
// 1.7e-7 evaluated in fp32).  Where both passes are bound by VALU issue, its nine fmas, which
// pair with other waves' instructions, cost less than a logarithm and a reciprocal, which do not:
// 32768 x 5120 x 16 890 -> 875 us, 9001 x 2048 x 16 146 -> 139.
__device__ __forceinline__ float softplus_poly(float v) {
  const float e = fast_exp2(-fabsf(v) * kLog2e);
  float p = 0.00519541185349226f;
  p = __builtin_fmaf(p, e, -0.02926170453429222f);
  p = __builtin_fmaf(p, e, 0.07763569802045822f);
  p = __builtin_fmaf(p, e, -0.1359216272830963f);
  p = __builtin_fmaf(p, e, 0.19059711694717407f);
  p = __builtin_fmaf(p, e, -0.24826765060424805f);
  p = __builtin_fmaf(p, e, 0.33316320180892944f);
  p = __builtin_fmaf(p, e, -0.4999932646751404f);
  p = __builtin_fmaf(p, e, 1.0f);
  return __builtin_fmaf(p, e, fmaxf(v, 0.0f));
}

// HAS_Z, YB (y is bf16): pass 2 only.
template <int NS, bool BF16, int PASS, int FL, bool HAS_Z, bool YB>
__global__ __launch_bounds__(128, pscan_min_waves(NS)) void packed_scan_kernel(
    const char* __restrict__ x, const char* __restrict__ delta, const float* __restrict__ A,
    const char* __restrict__ Bm, const char* __restrict__ Cm, const float* __restrict__ Dsk,
    const char* __restrict__ z, const float* __restrict__ dbias, float* __restrict__ state,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ sidx, const uint8_t* __restrict__ init,
    char* __restrict__ y, float* __restrict__ ws_end /* pass 1 out */, float* __restrict__ ws_sum,
    float* __restrict__ ws_init, const float* __restrict__ ws_enter /* pass 2 in */, int32_t* __restrict__ ws_flag,
    PScanGeo g) {
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int PL = NS < 4 ? NS : 4;    // states of a row that one lane stages
  constexpr int TS = 64 * PL / NS;       // steps per row tile
  constexpr int RT = PASS == 2 ? 2 : 1;  // tensors staged: B (, C)
  constexpr int TF = 64 * PL;            // floats per tensor and tile
  constexpr int U = 2;                   // steps per load batch
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t lid = xcd_remap(blockIdx.x, gridDim.x);
  const int grp = (int)(lid % (uint32_t)g.nblk) * g.gpb + wave;
  const int chunk = (int)(lid / (uint32_t)g.nblk);
  if (grp >= g.ngroups) return;  // not a copy of the last group: slots are updated in place
  const int64_t D = g.D;
  const int d0 = grp * 64;
  // lanes past the last channel repeat it: equal values, duplicate stores by the same wave
  const int dc = min(d0 + lane, g.D - 1);
  const int loff = dc - d0;
  const int c0 = chunk * g.K;
  const int lo = max(cu[0], 0), hi = min(cu[g.nseq], g.tokens);

  __shared__ float lds[2][2 * RT * TF];  // [wave][buffer][tensor][steps x states]
  float* const lrows = lds[wave];

  float a2[NS], h[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) a2[n] = decay_rate(A[(int64_t)dc * NS + n]);
  const float dbv = ((FL & kFront) != 0 && dbias != nullptr) ? dbias[dc] : 0.0f;
  const float Dd = (PASS == 2 && Dsk != nullptr) ? Dsk[dc] : 0.0f;
  constexpr bool has_z = PASS == 2 && HAS_Z, yb = YB;
  const bool bcb = g.bc_bf16 != 0;
  float dsum = 0.0f;
  const int rstep = lane * PL / NS, rcol = lane * PL % NS;  // the row tile's piece of this lane

  auto slot_load = [&](int slot) {
    const float* p = state + ((int64_t)slot * D + dc) * NS;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = p[n];
  };

  // tokens [t, e) of one sequence, at most g.piece of them, on the states in h
  auto walk_piece = [&](int t, int e) {
    const int len = e - t;
    const __amdgpu_buffer_rsrc_t rx = pscan_rsrc(x + ((int64_t)t * g.sx + d0) * ES);
    const __amdgpu_buffer_rsrc_t rd = pscan_rsrc(delta + ((int64_t)t * g.sd + d0) * ES);
    const __amdgpu_buffer_rsrc_t rz = pscan_rsrc(has_z ? z + ((int64_t)t * g.sz + d0) * ES : x);
    const __amdgpu_buffer_rsrc_t ry = pscan_rsrc(PASS == 2 ? y + ((int64_t)t * D + d0) * (yb ? 2 : 4) : x);
    const int xs = (int)g.sx * ES, ds = (int)g.sd * ES, zs = (int)g.sz * ES, ys = g.D * (yb ? 2 : 4);
    const int vo = loff * ES;
    const int yvo = loff * (yb ? 2 : 4);
    Vec<false, PL> grb, grc;  // a row tile in flight: fp32, or bf16 in the first half
    auto rows_load = [&](int j) {
      const int64_t tk = min(t + j * TS + rstep, e - 1);
      if (bcb) {
        Vec<true, PL> v;
        v.load(Bm + (tk * g.sb + rcol) * 2);
#pragma unroll
        for (int i = 0; i < Vec<true, PL>::ND; ++i) grb.w[i] = v.w[i];
        if constexpr (RT == 2) {
          v.load(Cm + (tk * g.sc + rcol) * 2);
#pragma unroll
          for (int i = 0; i < Vec<true, PL>::ND; ++i) grc.w[i] = v.w[i];
        }
      } else {
        grb.load(Bm + (tk * g.sb + rcol) * 4);
        if constexpr (RT == 2) grc.load(Cm + (tk * g.sc + rcol) * 4);
      }
    };
    auto rows_put = [&](const Vec<false, PL>& r, float* p) {
      float v[PL];
      if (bcb) {
        Vec<true, PL> b;
#pragma unroll
        for (int i = 0; i < Vec<true, PL>::ND; ++i) b.w[i] = r.w[i];
#pragma unroll
        for (int i = 0; i < PL; ++i) v[i] = b.get(i);
      } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) v[i] = r.get(i);
      }
      if constexpr (PL == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) p[i] = v[i];
      }
    };
    auto rows_store = [&](int buf) {
      rows_put(grb, lrows + buf * (RT * TF) + lane * PL);
      if constexpr (RT == 2) rows_put(grc, lrows + buf * (RT * TF) + TF + lane * PL);
    };
    uint32_t xq[2][U], dq[2][U], zq[2][U];
    auto ld = [&](__amdgpu_buffer_rsrc_t r, int so) -> uint32_t {
      if (BF16) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, vo, so, 2);
      return __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, 2);
    };
    auto wid = [](uint32_t v) -> float { return pscan_f32(BF16 ? v << 16 : v); };
    auto load = [&](int slot, int t0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int q = min(t0 + i, len - 1);
        xq[slot][i] = ld(rx, q * xs);
        dq[slot][i] = ld(rd, q * ds);
        if constexpr (has_z) zq[slot][i] = ld(rz, q * zs);
      }
    };
    // One step, the states in groups with three phases separated by scheduling barriers that
    // only memory and scalar instructions may cross -- the exponents, the exps at a raised wave
    // priority, the updates -- so that the waves' plain VALU instructions meet and issue in
    // pairs (measured on the dense scan: selective_scan.hip).
    auto step = [&](uint32_t xr, uint32_t dr, uint32_t zr, int i) {
      const float* brow = lrows + ((i / TS) & 1) * (RT * TF) + (i & (TS - 1)) * NS;
      const float xv = wid(xr);
      const float dv = wid(dr) + dbv;
      const float dl = (FL & kSoftplus) != 0 ? softplus_poly(dv) : dv;
      const float dx = dl * xv;
      float y0 = Dd * xv, y1 = 0.0f;
      constexpr int GS = NS < 4 ? NS : (NS >= 8 && BF16 && PASS == 1) ? 8 : 4;
#pragma unroll
      for (int n0 = 0; n0 < NS; n0 += GS) {
        float bq[GS], cq[GS], arg[GS], ab[GS];
        if constexpr (GS >= 4) {
#pragma unroll
          for (int q = 0; q < GS / 4; ++q) {
            const float4 v = reinterpret_cast<const float4*>(brow + n0)[q];
            bq[4 * q] = v.x; bq[4 * q + 1] = v.y; bq[4 * q + 2] = v.z; bq[4 * q + 3] = v.w;
            if constexpr (PASS == 2) {
              const float4 c = reinterpret_cast<const float4*>(brow + TF + n0)[q];
              cq[4 * q] = c.x; cq[4 * q + 1] = c.y; cq[4 * q + 2] = c.z; cq[4 * q + 3] = c.w;
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < GS; ++k) {
            bq[k] = brow[n0 + k];
            if constexpr (PASS == 2) cq[k] = brow[TF + n0 + k];
          }
        }
#pragma unroll
        for (int k = 0; k < GS; ++k) arg[k] = dl * a2[n0 + k];
        __builtin_amdgcn_sched_barrier(0x14);
        __builtin_amdgcn_s_setprio(2);
#pragma unroll
        for (int k = 0; k < GS; ++k) ab[k] = fast_exp2(arg[k]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0x14);
#pragma unroll
        for (int k = 0; k < GS; ++k) {
          const int n = n0 + k;
          h[n] = __builtin_fmaf(ab[k], h[n], dx * bq[k]);
          if constexpr (PASS == 2) {
            if (n & 1) y1 = __builtin_fmaf(cq[k], h[n], y1);
            else y0 = __builtin_fmaf(cq[k], h[n], y0);
          }
        }
        __builtin_amdgcn_sched_barrier(0x14);
      }
      if constexpr (PASS == 1) {
        dsum += dl;
        asm volatile("" ::"v"(dsum));  // needed here, not at the end of the unrolled tile
      } else {
        float out = y0 + y1;
        if constexpr (has_z) out *= silu(wid(zr));
        if constexpr (yb) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)vec_bf16_pair(out, 0.0f), ry, yvo, i * ys, 2);
        else __builtin_amdgcn_raw_buffer_store_b32(pscan_u32(out), ry, yvo, i * ys, 2);
      }
    };
    load(0, 0);
    rows_load(0);
    rows_store(0);
    rows_load(1);
    int t0 = 0;
    for (; t0 + TS <= len; t0 += TS) {
#pragma unroll 1
      for (int q = 0; q < TS; q += 2 * U) {
        load(1, t0 + q + U);
#pragma unroll
        for (int i = 0; i < U; ++i) step(xq[0][i], dq[0][i], zq[0][i], t0 + q + i);
        load(0, t0 + q + 2 * U);
#pragma unroll
        for (int i = 0; i < U; ++i) step(xq[1][i], dq[1][i], zq[1][i], t0 + q + U + i);
      }
      rows_store((t0 / TS + 1) & 1);
      rows_load(t0 / TS + 2);
    }
    for (; t0 < len; t0 += 2 * U) {  // fewer than TS steps left, all in the tile now in LDS
      load(1, t0 + U);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (t0 + i < len) step(xq[0][i], dq[0][i], zq[0][i], t0 + i);
      load(0, t0 + 2 * U);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (t0 + U + i < len) step(xq[1][i], dq[1][i], zq[1][i], t0 + U + i);
    }
  };

  auto walk = [&](int t, int e) {
    for (; t < e; t += g.piece) walk_piece(t, min(t + g.piece, e));
  };

  if constexpr (PASS == 1) {
    const int tend = c0 + g.K;
    int flag = 0;  // 0: no sequence runs across this chunk's end; 1: one from before it; 2: one that begins in it
    if (tend > lo && tend < hi) {
      const int s = min(max(find_seq(cu, g.nseq, tend - 1, lane), 0), g.nseq - 1);
      if (min(cu[s + 1], hi) > tend) {
        const int beg = min(max(cu[s], 0), tend);
        flag = beg >= c0 ? 2 : 1;
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = 0.0f;
        const int slot = sidx != nullptr ? sidx[s] : s;
        if (flag == 2 && state != nullptr && (unsigned)slot < (unsigned)g.slots && init != nullptr && init[s] != 0) {
          slot_load(slot);
          // kept for pass 2: the slot itself is overwritten there, by another chunk
#pragma unroll
          for (int n = 0; n < NS; ++n) ws_init[((int64_t)chunk * NS + n) * D + dc] = h[n];
        }
        walk(max(beg, c0), tend);
        ws_sum[(int64_t)chunk * D + dc] = dsum;
#pragma unroll
        for (int n = 0; n < NS; ++n) ws_end[((int64_t)chunk * NS + n) * D + dc] = h[n];
      }
    }
    if (grp == 0 && lane == 0) ws_flag[chunk] = flag;
  } else {
    int t = max(c0, lo);
    const int tend = min(c0 + g.K, hi);
    if (t >= tend) return;
    int s = min(max(find_seq(cu, g.nseq, t, lane), 0), g.nseq - 1);
    while (t < tend) {
      const int end = min(cu[s + 1], hi);
      if (end <= t) {  // past this sequence (or an empty one)
        if (++s >= g.nseq) break;
        continue;
      }
      const int slot = sidx != nullptr ? sidx[s] : s;
      const bool kept = state != nullptr && (unsigned)slot < (unsigned)g.slots;
      if (began_before(cu[s], c0)) {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = ws_enter[((int64_t)chunk * NS + n) * D + dc];
      } else if (kept && init != nullptr && init[s] != 0) {
        if (end > tend) {
#pragma unroll
          for (int n = 0; n < NS; ++n) h[n] = ws_init[((int64_t)chunk * NS + n) * D + dc];
        } else {
          slot_load(slot);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = 0.0f;
      }
      const int e = min(end, tend);
      walk(t, e);
      if (e == end && kept) {
        float* p = state + ((int64_t)slot * D + dc) * NS;
#pragma unroll
        for (int n = 0; n < NS; ++n) p[n] = h[n];
      }
      t = e;
    }
  }
}

template <int NS, bool BF16, int FL>
static hipError_t run_pscan(const PackedScanArgs& a, const PackedScanPlan& pl, hipStream_t stream) {
  PScanGeo g{};
  g.sx = a.sx;
  g.sd = a.sd;
  g.sz = a.sz;
  g.sb = a.sb;
  g.sc = a.sc;
  g.tokens = (int)a.tokens;
  g.nseq = (int)a.nseq;
  g.slots = (int)a.slots;
  g.D = (int)a.dim;
  g.K = (int)pl.K;
  g.ngroups = (int)((a.dim + 63) / 64);
  g.gpb = std::min(2, g.ngroups);
  g.nblk = (g.ngroups + g.gpb - 1) / g.gpb;
  const int64_t widest = std::max({a.sx, a.sd, a.sz, a.dim, (int64_t)1});
  g.piece = (int)std::min<int64_t>((((int64_t)1 << 28) / widest) & ~(int64_t)3, 1 << 28);  // strides <= 2^24: 16 at least
  g.bc_bf16 = a.bc_bf16;
  char* ws = static_cast<char*>(a.workspace);
  float* w_end = reinterpret_cast<float*>(ws + pl.off_end);
  float* w_sum = reinterpret_cast<float*>(ws + pl.off_sum);
  float* w_init = reinterpret_cast<float*>(ws + pl.off_init);
  float* w_enter = reinterpret_cast<float*>(ws + pl.off_enter);
  int32_t* w_flag = reinterpret_cast<int32_t*>(ws + pl.off_flag);
  const dim3 block(64u * g.gpb);
  if (pl.chunks > 1) {
    hipLaunchKernelGGL((packed_scan_kernel<NS, BF16, 1, FL, false, false>), dim3((unsigned)((int64_t)g.nblk * (pl.chunks - 1))), block, 0,
                       stream, (const char*)a.x, (const char*)a.delta, a.A, (const char*)a.B, (const char*)a.C, a.Dsk,
                       (const char*)a.z, a.delta_bias, a.state, a.cu, a.sidx, a.init, (char*)a.y, w_end, w_sum, w_init,
                       w_enter, w_flag, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_pscan_carry(a.A, w_end, w_sum, w_flag, w_enter, NS, (int)a.dim, pl.chunks, stream);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)((int64_t)g.nblk * pl.chunks));
#define SSS_PASS2(HZ, YB)                                                                                             \
  hipLaunchKernelGGL((packed_scan_kernel<NS, BF16, 2, FL, HZ, YB>), grid, block, 0, stream, (const char*)a.x,         \
                     (const char*)a.delta, a.A, (const char*)a.B, (const char*)a.C, a.Dsk, (const char*)a.z,          \
                     a.delta_bias, a.state, a.cu, a.sidx, a.init, (char*)a.y, w_end, w_sum, w_init, w_enter, w_flag, g)
  if (a.z != nullptr && a.y_bf16) SSS_PASS2(true, true);
  else if (a.z != nullptr) SSS_PASS2(true, false);
  else if (a.y_bf16) SSS_PASS2(false, true);
  else SSS_PASS2(false, false);
#undef SSS_PASS2
  return hipGetLastError();
}

template <int NS, bool BF16>
hipError_t run_pscan_front(const PackedScanArgs& a, const PackedScanPlan& pl, hipStream_t stream) {
  // without a bias, kFront adds zero
  return a.softplus ? run_pscan<NS, BF16, kFront | kSoftplus>(a, pl, stream) : run_pscan<NS, BF16, kFront>(a, pl, stream);
}

// compiled once per state count (SSS_INST_NS) and once for the host part
#ifdef SSS_INST_NS
template hipError_t run_pscan_front<SSS_INST_NS, false>(const PackedScanArgs&, const PackedScanPlan&, hipStream_t);
template hipError_t run_pscan_front<SSS_INST_NS, true>(const PackedScanArgs&, const PackedScanPlan&, hipStream_t);
#else
#define SSS_EXTERN_PSCAN(N)                                                                                         \
  extern template hipError_t run_pscan_front<N, false>(const PackedScanArgs&, const PackedScanPlan&, hipStream_t);  \
  extern template hipError_t run_pscan_front<N, true>(const PackedScanArgs&, const PackedScanPlan&, hipStream_t);
SSS_EXTERN_PSCAN(1)
SSS_EXTERN_PSCAN(2)
SSS_EXTERN_PSCAN(4)
SSS_EXTERN_PSCAN(8)
SSS_EXTERN_PSCAN(16)
SSS_EXTERN_PSCAN(32)
SSS_EXTERN_PSCAN(64)
#undef SSS_EXTERN_PSCAN

// One thread per (n, d) and range of chunks.  A chain is a run of chunks that one sequence
// crosses: it starts at a chunk with flag 2 and goes on over those with flag 1.  The thread
// follows the chains that start in its range, past the range's end where they reach further,
// so that the sequences of a batch are composed in parallel.
constexpr int kPCarryBatch = 16;
static __global__ __launch_bounds__(256) void pscan_carry_kernel(const float* __restrict__ A,
                                                                 const float* __restrict__ ends,
                                                                 const float* __restrict__ sums,
                                                                 const int32_t* __restrict__ flags,
                                                                 float* __restrict__ enter, int N, int D, int last,
                                                                 int range) {
  const int64_t per = (int64_t)N * D;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= per) return;
  const int n = (int)(idx / D), d = (int)(idx - (int64_t)n * D);
  const float a2 = decay_rate(A[(int64_t)d * N + n]);
  const int r0 = (int)blockIdx.y * range, r1 = min(r0 + range, last);  // chunks 0..last-1 have flags
  float h = 0.0f;
  bool on = false;
  for (int c0 = r0; c0 < last; c0 += kPCarryBatch) {
    if (c0 >= r1 && !on) return;
    int fl[kPCarryBatch], any = 0;
#pragma unroll
    for (int i = 0; i < kPCarryBatch; ++i) {
      fl[i] = c0 + i < last ? flags[c0 + i] : 0;
      any |= fl[i];
    }
    if (any == 0) {  // only short sequences here
      on = false;
      continue;
    }
    // loaded without regard to the flags, so that all of the batch is in flight together; where
    // a flag is 0 nothing was written, and nothing is used
    float st[kPCarryBatch], ds[kPCarryBatch];
#pragma unroll
    for (int i = 0; i < kPCarryBatch; ++i) {
      const int64_t c = min(c0 + i, last - 1);
      st[i] = ends[c * per + idx];
      ds[i] = sums[c * D + d];
    }
#pragma unroll
    for (int i = 0; i < kPCarryBatch; ++i) {
      const int c = c0 + i;
      if (fl[i] == 2) {
        on = c < r1;  // a chain that starts past the range is another's
        h = st[i];
      } else if (fl[i] == 1) {
        h = __builtin_fmaf(fast_exp2(a2 * ds[i]), h, st[i]);
      } else {
        on = false;
      }
      if (on) enter[(int64_t)(c + 1) * per + idx] = h;
    }
  }
}

hipError_t launch_pscan_carry(const float* A, const float* ends, const float* sums, const int32_t* flags, float* enter,
                              int dstate, int dim, int chunks, hipStream_t stream) {
  const int64_t per = (int64_t)dstate * dim;
  const int last = chunks - 1;
  const int ranges = std::max(1, std::min(8, last / 4));
  const int range = (last + ranges - 1) / ranges;
  hipLaunchKernelGGL(pscan_carry_kernel, dim3((unsigned)((per + 255) / 256), (unsigned)ranges), dim3(256), 0, stream, A,
                     ends, sums, flags, enter, dstate, dim, last, range);
  return hipGetLastError();
}

static size_t pscan_align(size_t v) { return (v + 255) / 256 * 256; }

PackedScanPlan plan_packed_scan(int64_t tokens, int64_t dim, int64_t dstate, int num_cus) {
  PackedScanPlan pl{};
  const int64_t groups = (dim + 63) / 64;
  // Waves (one per channel group and chunk) that the device holds at once in pass 2.  All waves
  // take about as long, so that a launch of one or two full rounds wastes nothing, and one of
  // a little more than a round nearly half: 9001 tokens x 2048 x 16 takes 135 us in 126 chunks (one
  // round), 153 in 141; 32768 x 5120 x 16 975 us in 51 (one), 906 in 102 (two), 1051 in 52.
  const int64_t simds = (int64_t)std::max(num_cus, 1) * 4;
  const int64_t round = std::max<int64_t>(1, simds * pscan_min_waves((int)dstate) / groups);  // chunks
  // two rounds of chunks of 64 tokens at least (16384 x 1024 x 8: 90 us in one round of 64 tokens,
  // 98 in two of 32), else one of 32; 16 where 32 would leave most SIMDs idle (300 x 1024 x 16:
  // 23 us, 31 with 32)
  int64_t S = tokens >= 2 * round * 64 ? 2 * round : round;
  const int64_t shortest = groups * ((tokens + 31) / 32) * 2 >= simds ? 32 : 16;
  S = std::min<int64_t>(S, std::max<int64_t>(1, tokens / shortest));
  const int forced = env_int("SSS_FORCE_SEGMENTS", 0);
  if (forced > 0) S = std::min<int64_t>(forced, tokens);
  const int64_t K = std::max<int64_t>(1, (tokens + S - 1) / S);
  pl.K = K;
  pl.chunks = (int)((tokens + K - 1) / K);
  if (pl.chunks > 1) {
    const size_t st = pscan_align((size_t)pl.chunks * dim * dstate * 4);
    pl.off_end = 0;
    pl.off_init = st;
    pl.off_enter = 2 * st;
    pl.off_sum = 3 * st;
    pl.off_flag = pl.off_sum + pscan_align((size_t)pl.chunks * dim * 4);
    pl.ws_total = pl.off_flag + pscan_align((size_t)pl.chunks * 4);
  }
  return pl;
}

template <bool BF16>
static hipError_t dispatch_pscan(const PackedScanArgs& a, const PackedScanPlan& pl, hipStream_t stream) {
  switch (a.dstate) {
    case 1: return run_pscan_front<1, BF16>(a, pl, stream);
    case 2: return run_pscan_front<2, BF16>(a, pl, stream);
    case 4: return run_pscan_front<4, BF16>(a, pl, stream);
    case 8: return run_pscan_front<8, BF16>(a, pl, stream);
    case 16: return run_pscan_front<16, BF16>(a, pl, stream);
    case 32: return run_pscan_front<32, BF16>(a, pl, stream);
    case 64: return run_pscan_front<64, BF16>(a, pl, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_packed_scan(const PackedScanArgs& a, const PackedScanPlan& pl, hipStream_t stream) {
  return a.bf16 ? dispatch_pscan<true>(a, pl, stream) : dispatch_pscan<false>(a, pl, stream);
}
#endif  // SSS_INST_NS

}  // namespace sss

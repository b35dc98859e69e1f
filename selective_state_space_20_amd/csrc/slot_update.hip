// slot_update.hip -- gfx950 kernel of one decode step of the selective scan on states kept in
// cache slots, through the delta front end.
//
//   dt = delta[b,d], or + bias[d], or softplus of that;  h = state[slot_b, d, :]
//   h[n] = exp(dt A[d,n]) h[n] + dt B[b,n] x[b,d]                       (in place)
//   y[b,d] = (sum_n C[b,n] h[n] + D[d] x[b,d]) silu(z[b,d])
// A row whose index is no slot (negative) starts from zero and keeps nothing.
//
// Bound by moving the states, 8 bytes per state and row (256 rows x 5120 x 16: 179 MB in 35-36 us,
// 5 TB/s), as state_update.hip, whose mapping it shares: lanes walk (d, n) in memory order with four states each, R rows per thread with all
// their loads in flight.
#include "front.h"
#include "vec.h"
#include "kernels.h"

#include <algorithm>

namespace sss {

template <int CTRL>
__device__ __forceinline__ float slot_dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// sum over each group of LPC adjacent lanes (a power of two up to 16), in every lane of it
template <int LPC>
__device__ __forceinline__ float slot_sum(float p) {
  if constexpr (LPC >= 2) p += slot_dpp<0xB1>(p);    // quad_perm [1,0,3,2]
  if constexpr (LPC >= 4) p += slot_dpp<0x4E>(p);    // quad_perm [2,3,0,1]
  if constexpr (LPC >= 8) p += slot_dpp<0x141>(p);   // row_half_mirror
  if constexpr (LPC >= 16) p += slot_dpp<0x140>(p);  // row_mirror
  return p;
}

struct SlotGeo {
  int64_t sx, sd, sz, sb, sc;  // elements between rows
  int rows, slots, D;
  unsigned bpr;  // workgroups per group of R rows
  int bc_bf16, y_bf16, front, softplus;
};

template <int NS, bool BF16, int R>
__global__ __launch_bounds__(256) void slot_update_kernel(const char* __restrict__ x, const char* __restrict__ delta,
                                                          const float* __restrict__ A, const char* __restrict__ Bm,
                                                          const char* __restrict__ Cm, const float* __restrict__ Dsk,
                                                          const char* __restrict__ z, const float* __restrict__ dbias,
                                                          float* __restrict__ state, const int32_t* __restrict__ sidx,
                                                          char* __restrict__ y, SlotGeo g) {
  constexpr int PL = NS >= 4 ? 4 : NS;
  constexpr int LPC = NS / PL;
  constexpr int ES = BF16 ? 2 : 4;
  const unsigned rg = blockIdx.x / g.bpr;
  const int li = (int)(blockIdx.x - rg * g.bpr) * 256 + (int)threadIdx.x;  // lane index within a row
  // lanes past the row's end work on its last channel, so that whole groups take part in the
  // lane sums, and store nothing
  const int lanes = g.D * LPC;
  const bool live = li < lanes;
  const int d = (live ? li : lanes - 1) / LPC;
  const int j = (live ? li : lanes - 1) - d * LPC;

  Vec<false, PL> av;
  av.load(A + (int64_t)d * NS + j * PL);
  const float dd = Dsk != nullptr ? Dsk[d] : 0.0f;
  const float bias = dbias != nullptr ? dbias[d] : 0.0f;
  const bool has_z = z != nullptr;

  Vec<false, PL> hv[R];
  Vec<BF16, 1> xv[R], dv[R], zv[R];
  float bv[R][PL], cv[R][PL];
  int slot[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = (int)rg * R + r;
    slot[r] = row < g.rows ? (sidx != nullptr ? sidx[row] : row) : -1;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = min((int)rg * R + r, g.rows - 1);
    if ((unsigned)slot[r] < (unsigned)g.slots) hv[r].template load<true>(state + ((int64_t)slot[r] * g.D + d) * NS + j * PL);
    else hv[r].zero();
    xv[r].load(x + (row * g.sx + d) * ES);
    dv[r].load(delta + (row * g.sd + d) * ES);
    if (has_z) zv[r].load(z + (row * g.sz + d) * ES);
    if (g.bc_bf16) {
      Vec<true, PL> b, c;
      b.load(Bm + (row * g.sb + j * PL) * 2);
      c.load(Cm + (row * g.sc + j * PL) * 2);
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        bv[r][i] = b.get(i);
        cv[r][i] = c.get(i);
      }
    } else {
      Vec<false, PL> b, c;
      b.load(Bm + (row * g.sb + j * PL) * 4);
      c.load(Cm + (row * g.sc + j * PL) * 4);
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        bv[r][i] = b.get(i);
        cv[r][i] = c.get(i);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = (int)rg * R + r;
    const float xf = xv[r].get(0);
    float dt = dv[r].get(0);
    if (g.front) dt += bias;
    if (g.softplus) dt = softplus_f(dt);
    const float dx = dt * xf;
    float hn[PL], part = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const float a2 = decay_rate(av.get(i));
      hn[i] = __builtin_fmaf(fast_exp2(dt * a2), hv[r].get(i), dx * bv[r][i]);
      part = __builtin_fmaf(cv[r][i], hn[i], part);
    }
    if (live && (unsigned)slot[r] < (unsigned)g.slots) {
      Vec<false, PL> o;
      o.set(hn);
      o.store(state + ((int64_t)slot[r] * g.D + d) * NS + j * PL);
    }
    part = slot_sum<LPC>(part);
    if (live && row < g.rows && j == 0) {
      float out[1] = {__builtin_fmaf(dd, xf, part)};
      if (has_z) out[0] *= silu(zv[r].get(0));
      const int64_t i = (int64_t)row * g.D + d;
      if (g.y_bf16) {
        Vec<true, 1> o;
        o.set(out);
        o.store(y + i * 2);
      } else {
        *reinterpret_cast<float*>(y + i * 4) = out[0];
      }
    }
  }
}

template <int NS, bool BF16, int R>
static hipError_t run_slots_r(const PackedScanArgs& a, hipStream_t stream) {
  constexpr int LPC = NS >= 4 ? NS / 4 : 1;
  SlotGeo g{};
  g.sx = a.sx;
  g.sd = a.sd;
  g.sz = a.sz;
  g.sb = a.sb;
  g.sc = a.sc;
  g.rows = (int)a.tokens;
  g.slots = (int)a.slots;
  g.D = (int)a.dim;
  g.bpr = (unsigned)((a.dim * LPC + 255) / 256);
  g.bc_bf16 = a.bc_bf16;
  g.y_bf16 = a.y_bf16;
  g.front = a.delta_bias != nullptr;
  g.softplus = a.softplus;
  const dim3 grid((unsigned)(g.bpr * ((a.tokens + R - 1) / R))), block(256);
  hipLaunchKernelGGL((slot_update_kernel<NS, BF16, R>), grid, block, 0, stream, (const char*)a.x, (const char*)a.delta,
                     a.A, (const char*)a.B, (const char*)a.C, a.Dsk, (const char*)a.z, a.delta_bias, a.state, a.sidx,
                     (char*)a.y, g);
  return hipGetLastError();
}

// Two rows per thread: 37 us at 256 rows x 5120 x 16 with the states loaded past the caches and
// stored through them, against 43 with four rows and cached loads, 39 with four and past the
// caches both ways, 40 with one row.
constexpr int kSlotRows = 2;

template <int NS, bool BF16>
static hipError_t run_slots(const PackedScanArgs& a, hipStream_t stream) {
  return run_slots_r<NS, BF16, kSlotRows>(a, stream);
}

// as run_slots_r: four states per lane (or all of fewer), whole workgroups per group of rows
double slot_update_threads(int64_t rows, int64_t dim, int64_t dstate) {
  const int64_t lanes = dim * std::max<int64_t>(dstate / 4, 1);
  return (double)((rows + kSlotRows - 1) / kSlotRows) * (double)((lanes + 255) / 256) * 256.0;
}

template <bool BF16>
static hipError_t dispatch_slots(const PackedScanArgs& a, hipStream_t stream) {
  switch (a.dstate) {
    case 1: return run_slots<1, BF16>(a, stream);
    case 2: return run_slots<2, BF16>(a, stream);
    case 4: return run_slots<4, BF16>(a, stream);
    case 8: return run_slots<8, BF16>(a, stream);
    case 16: return run_slots<16, BF16>(a, stream);
    case 32: return run_slots<32, BF16>(a, stream);
    case 64: return run_slots<64, BF16>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_slot_update(const PackedScanArgs& a, hipStream_t stream) {
  return a.bf16 ? dispatch_slots<true>(a, stream) : dispatch_slots<false>(a, stream);
}

}  // namespace sss

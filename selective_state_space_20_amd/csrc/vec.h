// vec.h -- V adjacent elements of one lane, bf16 or fp32, moved as one wide access, and the
// search of a packed batch's sequence boundaries (HIP, gfx950).
#pragma once
#include "common.h"

namespace sss {

// Wide accesses at element alignment: rows of an odd length, or halves of a projection's rows,
// start at any element.  gfx950 runs with unaligned global accesses enabled (the compiler
// emits one wide load or store for these types), so that no narrower path is needed.
typedef uint32_t vec_u1 __attribute__((aligned(2)));
typedef uint32_t vec_u2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t vec_u4 __attribute__((ext_vector_type(4), aligned(2)));

typedef __bf16 vec_bf2 __attribute__((ext_vector_type(2)));
typedef float vec_f2 __attribute__((ext_vector_type(2)));

// two fp32 -> two bf16 in one dword (low half = a), rounded to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t vec_bf16_pair(float a, float b) {
  const vec_f2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, vec_bf2));
}

// A row's address, the same in the whole wave, and a lane's byte offset in it: kept apart (a
// scalar register pair and one vector register), so that an access needs no vector address
// arithmetic.  Left alone the compiler folds both into a 64-bit vector address per access.
typedef __attribute__((address_space(1))) char* row_ptr;
__device__ __forceinline__ row_ptr row_at(const void* base, int64_t bytes) {
  row_ptr p = (row_ptr)(const_cast<char*>(static_cast<const char*>(base)) + bytes);
  asm volatile("" : "+s"(p));
  return p;
}
__device__ __forceinline__ uint32_t lane_at(uint32_t off) {
  asm volatile("" : "+v"(off));
  return off;
}

// One access of 2, 4, 8 or 16 bytes through either kind of pointer.  The types are spelled out:
// as a template argument a type loses its alignment, and the compiler then takes rows that are
// the same for all lanes through scalar loads, which drop an address's low two bits.
#define SSS_VEC_ACCESS(NAME, T, PTR, AS)                                    \
  template <bool NT>                                                        \
  __device__ __forceinline__ T vec_get##NAME(PTR p) {                       \
    if constexpr (NT) return __builtin_nontemporal_load((const AS T*)p);    \
    else return *(const AS T*)p;                                            \
  }                                                                         \
  template <bool NT>                                                        \
  __device__ __forceinline__ void vec_put##NAME(PTR p, T v) {               \
    if constexpr (NT) __builtin_nontemporal_store(v, (AS T*)p);             \
    else *(AS T*)p = v;                                                     \
  }
#define SSS_VEC_AS1 __attribute__((address_space(1)))
SSS_VEC_ACCESS(2, uint16_t, char*, )
SSS_VEC_ACCESS(4, vec_u1, char*, )
SSS_VEC_ACCESS(8, vec_u2, char*, )
SSS_VEC_ACCESS(16, vec_u4, char*, )
SSS_VEC_ACCESS(2, uint16_t, row_ptr, SSS_VEC_AS1)
SSS_VEC_ACCESS(4, vec_u1, row_ptr, SSS_VEC_AS1)
SSS_VEC_ACCESS(8, vec_u2, row_ptr, SSS_VEC_AS1)
SSS_VEC_ACCESS(16, vec_u4, row_ptr, SSS_VEC_AS1)
#undef SSS_VEC_ACCESS
#undef SSS_VEC_AS1

template <bool BF16, int V>
struct Vec {
  static constexpr int ES = BF16 ? 2 : 4;       // bytes per element
  static constexpr int VB = V * ES;             // bytes per lane
  static constexpr int ND = VB >= 4 ? VB / 4 : 1;
  uint32_t w[ND];  // raw bits: widened only when read, so that loads stay in flight

  // NT: streamed data that nothing reads again soon.  P: a generic pointer, or a row_ptr + offset
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* p) {
    load_as<NT, char*>(const_cast<char*>(static_cast<const char*>(p)));
  }
  template <bool NT = false>
  __device__ __forceinline__ void load(row_ptr p, uint32_t off) {
    load_as<NT, row_ptr>(p + off);
  }
  template <bool NT, typename P>
  __device__ __forceinline__ void load_as(P p) {
    if constexpr (VB == 2) {
      w[0] = vec_get2<NT>(p);
    } else if constexpr (VB == 4) {
      w[0] = vec_get4<NT>(p);
    } else if constexpr (VB == 8) {
      const vec_u2 v = vec_get8<NT>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      static_assert(VB % 16 == 0, "vector bytes");
#pragma unroll
      for (int i = 0; i < VB / 16; ++i) {
        const vec_u4 v = vec_get16<NT>(p + 16 * i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < ND; ++i) w[i] = 0u;
  }
  // element c widened to fp32
  __device__ __forceinline__ float get(int c) const {
    if constexpr (BF16) {
      const uint32_t d = w[c >> 1];
      return __builtin_bit_cast(float, (c & 1) ? (d & 0xFFFF0000u) : (d << 16));
    } else {
      return __builtin_bit_cast(float, w[c]);
    }
  }
  // from fp32, rounded once to nearest even in bf16
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (BF16) {
      if constexpr (V == 1) {
        w[0] = vec_bf16_pair(v[0], 0.0f) & 0xFFFFu;
      } else {
#pragma unroll
        for (int c = 0; c < V; c += 2) w[c >> 1] = vec_bf16_pair(v[c], v[c + 1]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) w[c] = __builtin_bit_cast(uint32_t, v[c]);
    }
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(void* p) const {
    store_as<NT, char*>(static_cast<char*>(p));
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(row_ptr p, uint32_t off) const {
    store_as<NT, row_ptr>(p + off);
  }
  template <bool NT, typename P>
  __device__ __forceinline__ void store_as(P p) const {
    if constexpr (VB == 2) {
      vec_put2<NT>(p, (uint16_t)w[0]);
    } else if constexpr (VB == 4) {
      vec_put4<NT>(p, w[0]);
    } else if constexpr (VB == 8) {
      const vec_u2 v = {w[0], w[1]};
      vec_put8<NT>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < VB / 16; ++i) {
        const vec_u4 v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        vec_put16<NT>(p + 16 * i, v);
      }
    }
  }
  // elements skip..V-1 only (skip 0: one wide store; skip V: nothing)
  template <bool NT = false>
  __device__ __forceinline__ void store_from(void* p, int skip) const {
    if (skip == 0) {
      store<NT>(p);
    } else {
      part_as(static_cast<char*>(p), skip);
    }
  }
  template <bool NT = false>
  __device__ __forceinline__ void store_from(row_ptr p, uint32_t off, int skip) const {
    if (skip == 0) {
      store<NT>(p, off);
    } else {
      part_as(p + off, skip);
    }
  }
  template <typename P>
  __device__ __forceinline__ void part_as(P p, int skip) const {
#pragma unroll
    for (int c = 1; c < V; ++c) {
      if (c < skip) continue;
      if constexpr (BF16) vec_put2<false>(p + 2 * c, (uint16_t)((c & 1) ? w[c >> 1] >> 16 : w[c >> 1]));
      else vec_put4<false>(p + 4 * c, w[c]);
    }
  }
};

// Packed sequences: the sequence that token t belongs to, i.e. the last s with cu[s] <= t
// among cu[0..nseq] (-1: before the first).  The whole wave searches: 64 boundaries per load,
// so that 64 sequences take one load and 4096 two.  Any contents of cu give a number in
// [-1, nseq].
// In two halves, so that the first load can be issued ahead of others: vector loads return in
// order, and waiting for this one does not wait for those after it.
struct SeqSearch {
  const int32_t* cu;
  int cnt, lane, first;
  __device__ __forceinline__ SeqSearch(const int32_t* cu_, int nseq, int lane_) : cu(cu_), cnt(nseq + 1), lane(lane_) {
    first = cu[min(lane * ((cnt + 63) >> 6), nseq)];
  }
  __device__ __forceinline__ int find(int t) const {
    int step = (cnt + 63) >> 6, lo = 0, n = cnt;
    int k = __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane * step < n && first <= t));
    while (step > 1) {
      if (k == 0) return lo - 1;
      lo += (k - 1) * step;
      n = min(step, n - (k - 1) * step);
      step = (n + 63) >> 6;
      const int i = lane * step;
      const bool le = i < n && cu[lo + i] <= t;
      k = __builtin_popcountll(__builtin_amdgcn_ballot_w64(le));
    }
    return lo - 1 + k;
  }
};
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int nseq, int t, int lane) {
  return SeqSearch(cu, nseq, lane).find(t);
}

}  // namespace sss

// api_util.h -- argument checks shared by the files of the C ABI (host only).
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace sss {

// Sizes in bytes with overflow checks; false when a product leaves [0, 2^62).
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > (int64_t(1) << 62) / a) return false;
  *out = a * b;
  return true;
}

inline bool overlap(const void* p, int64_t bytes, const void* q, int64_t qbytes) {
  if (p == nullptr || q == nullptr || bytes <= 0 || qbytes <= 0) return false;
  uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + (uintptr_t)qbytes && b < a + (uintptr_t)bytes;
}

inline bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned_to(const void* p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

// Bytes from the first to the last element of `rows` rows of `dim` elements, `stride` apart.
inline int64_t span(int64_t rows, int64_t stride, int64_t dim, int64_t es) {
  return rows < 1 ? 0 : ((rows - 1) * stride + dim) * es;
}

// The device memory that a call reads or writes: each argument once, with its bytes and the
// alignment its element type needs.  ok() is the overlap rule of every call: an output may
// not share memory with an input, another output or the workspace.
struct Regions {
  static constexpr int kMax = 24;
  const void* p[kMax];
  int64_t bytes[kMax];
  bool out[kMax];
  int n = 0;
  bool aligned = true;
  void add(const void* ptr, int64_t b, int64_t align, bool is_out) {
    if (ptr == nullptr) return;
    if (!aligned_to(ptr, align)) aligned = false;
    p[n] = ptr;
    bytes[n] = b;
    out[n++] = is_out;
  }
  void in(const void* ptr, int64_t b, int64_t align) { add(ptr, b, align, false); }
  void output(const void* ptr, int64_t b, int64_t align) { add(ptr, b, align, true); }
  bool ok() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((out[i] || out[j]) && overlap(p[i], bytes[i], p[j], bytes[j])) return false;
    return true;
  }
};

}  // namespace sss

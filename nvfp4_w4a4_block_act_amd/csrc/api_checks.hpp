// Argument checks shared by the entry points of the C ABI: size bounds, pointer
// alignment and buffer overlaps.  Host code only; nothing here calls HIP.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/nvfp4.h"

namespace nvfp4 {
namespace checks {

constexpr int64_t kMaxDim = (int64_t)1 << 31;  // kernel index math is 32-bit per dimension

// Leading dimensions are bounded like the other sizes, so that the extents
// (rows - 1) * ld + cols computed below stay far inside int64.
inline bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < kMaxDim; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A device buffer a call touches: base pointer and extent in bytes (0 = not
// touched by this call).
struct Buf {
  const void* p;
  size_t n;
};

inline bool overlap(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// No buffer a call writes overlaps another one it writes or one it reads
// (inputs may share memory with each other).
template <int NO, int NI>
inline bool disjoint(const Buf (&outs)[NO], const Buf (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return false;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}

// Every non-null pointer of the list is 16-byte aligned.
inline bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return false;
  return true;
}

inline nvfp4_status launched(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }

// Bytes spanned by `rows` rows of `cols` elements of `elem` bytes at row stride ld.
inline size_t extent(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  return (rows == 0 || cols == 0) ? 0 : (size_t)((rows - 1) * ld + cols) * elem;
}

}  // namespace checks
}  // namespace nvfp4

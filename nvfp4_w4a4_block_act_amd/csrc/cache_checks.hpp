// Checks of a paged cache's description, shared by the entry points that take one: sizes,
// strides, and that no two rows share memory.  Host code only; nothing here calls HIP.
#pragma once

#include <stdint.h>

#include <utility>

#include "api_checks.hpp"

namespace nvfp4 {
namespace checks {

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // cache strides, in elements: extents stay inside int64
constexpr int kMaxHeads = 1 << 16;
constexpr int64_t kMaxLen = (int64_t)1 << 30;     // token index plus a split's tokens stay inside int32
constexpr int64_t kMaxGroups = 1 << 22;  // workgroups of a launch: at most 2^32 threads

inline size_t cache_elem(const nvfp4_kv_cache& c) { return c.dtype == NVFP4_E4M3 ? 1 : 2; }

// Elements that the rows of one cache tensor span.
inline int64_t cache_span(const nvfp4_kv_cache& c) {
  return c.num_pages == 0 ? 0
                          : (c.num_pages - 1) * c.page_stride + (int64_t)(c.page_size - 1) * c.token_stride +
                                (int64_t)(c.kv_heads - 1) * c.head_stride + c.head_dim;
}

// The three axes that a row's place in a cache tensor has, by growing stride.
struct Axes {
  int64_t stride[3], count[3];
};
inline Axes axes_of(const nvfp4_kv_cache& c) {
  Axes a = {{c.head_stride, c.token_stride, c.page_stride}, {c.kv_heads, c.page_size, c.num_pages}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (a.stride[j] < a.stride[i]) {
        std::swap(a.stride[i], a.stride[j]);
        std::swap(a.count[i], a.count[j]);
      }
  return a;
}

// Rows of one tensor do not overlap: each axis steps over what the smaller ones span (an
// axis of one element has no stride).
inline bool rows_disjoint(const Axes& a, int64_t dim) {
  int64_t span = dim;
  for (int i = 0; i < 3; ++i) {
    if (a.count[i] <= 1) continue;
    if (a.stride[i] < span) return false;
    span += (a.count[i] - 1) * a.stride[i];
  }
  return true;
}

// Whether two rows of tensors `rest` elements apart, which differ by any steps along the
// axes up to `axis`, have an element in common.  Since an axis steps over what the smaller
// ones span, only the two steps on either side of `rest` come near enough.
inline bool rows_meet(const Axes& a, int64_t dim, int64_t rest, int axis) {
  if (axis < 0) return rest > -dim && rest < dim;
  if (a.count[axis] <= 1) return rows_meet(a, dim, rest, axis - 1);
  const int64_t most = a.count[axis] - 1, stride = a.stride[axis];
  const int64_t below = rest / stride - (rest % stride < 0 ? 1 : 0);
  for (const int64_t n : {below, below + 1})
    if (n >= -most && n <= most && rows_meet(a, dim, rest - n * stride, axis - 1)) return true;
  return false;
}

// No row of a tensor at x overlaps one of a tensor of the same shape at y (rows_disjoint
// holds): they may lie interleaved.
inline bool bases_disjoint(const nvfp4_kv_cache& c, const Axes& a, const void* x, const void* y) {
  if (c.num_pages == 0) return true;
  const uintptr_t k = reinterpret_cast<uintptr_t>(x), v = reinterpret_cast<uintptr_t>(y);
  const uintptr_t apart = (k < v ? v - k : k - v) / cache_elem(c);  // whole elements: both are aligned
  return apart >= (uintptr_t)1 << 60 || !rows_meet(a, c.head_dim, (int64_t)apart, 2);  // spans are below 2^58
}

inline bool tensors_disjoint(const nvfp4_kv_cache& c, const Axes& a) { return bases_disjoint(c, a, c.k, c.v); }

inline nvfp4_status check_cache(const nvfp4_kv_cache* c) {
  if (!c) return NVFP4_EINVAL;
  if (c->num_pages < 0 || c->page_size < 1 || c->kv_heads < 1) return NVFP4_EINVAL;
  if (c->dtype != NVFP4_BF16 && c->dtype != NVFP4_E4M3) return NVFP4_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ESHAPE;
  if (c->page_size % 16 != 0 || c->page_size > (1 << 20) || c->kv_heads > kMaxHeads || c->num_pages >= kMaxDim)
    return NVFP4_ESHAPE;
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < 0 || s >= kMaxStride) return NVFP4_ESHAPE;
  if (c->token_stride >= (1 << 26)) return NVFP4_ESHAPE;  // 16 rows within 32-bit byte offsets
  // (num_pages - 1) * page_stride must stay far inside int64
  if (c->num_pages > 1 && c->page_stride > ((int64_t)1 << 56) / c->num_pages) return NVFP4_ESHAPE;
  const Axes axes = axes_of(*c);
  if (!rows_disjoint(axes, c->head_dim)) return NVFP4_ESHAPE;
  if (c->num_pages > 0 && (!c->k || !c->v || c->k == c->v)) return NVFP4_EINVAL;
  if (c->dtype == NVFP4_E4M3 && (!c->k_amax || !c->v_amax)) return NVFP4_EINVAL;
  if (!all_aligned({c->k, c->v, c->k_amax, c->v_amax})) return NVFP4_EALIGN;
  const int64_t unit = 16 / (int64_t)cache_elem(*c);
  if (c->page_stride % unit || c->token_stride % unit || c->head_stride % unit) return NVFP4_EALIGN;
  return tensors_disjoint(*c, axes) ? NVFP4_OK : NVFP4_EINVAL;
}

}  // namespace checks
}  // namespace nvfp4

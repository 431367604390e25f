// Rows and pages of the paged key-value cache that move, in the caches of all layers at once.
//
// kv_compact: the accepted nodes of a drafted tree lie at rows ctx + path[i] of a sequence,
// and belong at ctx + i.  A destination may be another node's source, so a workgroup reads
// all pieces of its columns (a tensor's head: rows of one column only move within it) into
// registers before it writes any: 256 threads hold 8 pieces of 16 bytes each, which is a
// whole tree of 64 nodes of the widest row (512 bytes), or several heads of smaller ones.
// A workgroup whose sequence keeps every row where it is reads its path and ends.
//
// Bound by its launch and two chains of loads: 3.7 us alone for a chain of 8 in 16 layers,
// 5.3 us for 64 trees of 24 (4.3 MB).
//
// kv_copy_pages: a thread moves one piece of 16 bytes, 4 KB a workgroup, past the caches (the
// pages are more than they hold, or are not read again soon).  Bound by HBM: 96 pages of 16
// layers (403 MB read and written) take 69 us after other work and 68 back to back, 5.9 TB/s,
// where a library's copy of 1 GiB reaches 5.2.  With ordinary loads and stores 75 and 74,
// loads alone past the caches 76 and 62 (and more for 3 to 12 pages); four pieces a thread
// 80 and 78, eight 106, workgroups of 1024 threads 74.
#include <algorithm>

#include "common.hpp"
#include "drafts.hpp"

namespace nvfp4 {

constexpr int kMoveThreads = 256, kMovePieces = 8;

__host__ __device__ static inline int elem_size(const nvfp4_kv_cache& c) { return c.dtype == NVFP4_E4M3 ? 1 : 2; }

__global__ __launch_bounds__(kMoveThreads) void kv_compact_kernel(CompactArgs a, LayerCaches caches, int cols, int groups) {
  const nvfp4_kv_cache& c = caches.shape;
  const int part = blockIdx.x % groups, rest = blockIdx.x / groups;
  const int layer = rest % caches.layers, b = rest / caches.layers;
  const int es = elem_size(c), pieces = c.head_dim * es / 16;
  __shared__ int64_t from[NVFP4_MAX_NODES], to[NVFP4_MAX_NODES];
  __shared__ int moves;

  // rows that move, one after the other: byte offsets in a column
  if (threadIdx.x < 64) {
    const int i = threadIdx.x;
    const int count = min(max(a.counts[b], 0), a.nodes), ctx = a.lens[b];
    bool move = false;
    int64_t f = 0, t = 0;
    if (i < count) {
      const int j = a.path[(int64_t)b * a.nodes + i];
      const int64_t tokens = a.ldt * c.page_size, src = (int64_t)ctx + j, dst = (int64_t)ctx + i;
      if (j != i && j >= 0 && j < a.nodes && ctx >= 0 && src < tokens && dst < tokens) {
        const int ps = a.table[b * a.ldt + src / c.page_size], pd = a.table[b * a.ldt + dst / c.page_size];
        move = ps >= 0 && ps < c.num_pages && pd >= 0 && pd < c.num_pages;
        f = (ps * c.page_stride + src % c.page_size * c.token_stride) * es;
        t = (pd * c.page_stride + dst % c.page_size * c.token_stride) * es;
      }
    }
    const uint64_t all = __ballot(move);
    if (move) {
      const int at = __popcll(all & ((1ull << i) - 1));
      from[at] = f, to[at] = t;
    }
    if (i == 0) moves = __popcll(all);
  }
  __syncthreads();
  const int n = moves;
  if (n == 0) return;

  const int first = part * cols, last = min(first + cols, 2 * c.kv_heads);  // columns: k's heads, then v's
  const int total = (last - first) * n * pieces;
  u32x4_t held[kMovePieces];
  uint8_t* where[kMovePieces];
#pragma unroll
  for (int s = 0; s < kMovePieces; ++s) {
    const int p = threadIdx.x + s * kMoveThreads;
    where[s] = nullptr;
    if (p < total) {
      const int row = p / pieces, col = first + row / n, i = row % n;
      uint8_t* base = (col < c.kv_heads ? caches.k[layer] : caches.v[layer]) +
                      (int64_t)(col % c.kv_heads) * c.head_stride * es + p % pieces * 16;
      held[s] = *reinterpret_cast<const u32x4_t*>(base + from[i]);
      where[s] = base + to[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kMovePieces; ++s)
    if (where[s]) *reinterpret_cast<u32x4_t*>(where[s]) = held[s];
}

hipError_t launch_kv_compact(const CompactArgs& a, const LayerCaches& caches, hipStream_t stream) {
  const int pieces = caches.shape.head_dim * elem_size(caches.shape) / 16;
  const int cols = std::min(2 * caches.shape.kv_heads, kMoveThreads * kMovePieces / (a.nodes * pieces));
  const int groups = (2 * caches.shape.kv_heads + cols - 1) / cols;
  kv_compact_kernel<<<dim3((unsigned)((int64_t)a.B * caches.layers * groups)), kMoveThreads, 0, stream>>>(a, caches, cols, groups);
  return hipGetLastError();
}

constexpr int kCopyThreads = 256;

// Runs of a page: rows that follow each other without a gap count as one.
PageShape page_shape(const nvfp4_kv_cache& c) {
  const int es = elem_size(c);
  int64_t stride[2] = {c.head_stride * es, c.token_stride * es}, count[2] = {c.kv_heads, c.page_size};
  const int in = count[0] > 1 && (count[1] <= 1 || stride[0] <= stride[1]) ? 0 : 1, out = 1 - in;
  PageShape p = {c.head_dim * es, count[in], stride[in], count[out], stride[out]};
  if (p.mid == 1 || p.mid_stride == p.run) p.run *= p.mid, p.mid = 1;
  if (p.mid == 1) {
    if (p.outer == 1 || p.outer_stride == p.run) p.run *= p.outer, p.outer = 1;
    p.mid = p.outer, p.mid_stride = p.outer_stride, p.outer = 1, p.outer_stride = 0;
  }
  return p;
}

static int64_t page_pieces(const PageShape& p) { return p.run / 16 * p.mid * p.outer; }

int64_t copy_groups(const PageShape& p) { return (page_pieces(p) + kCopyThreads - 1) / kCopyThreads; }

template <bool WHOLE>
__global__ __launch_bounds__(kCopyThreads) void kv_copy_pages_kernel(const int32_t* src, const int32_t* dst,
                                                                    LayerCaches caches, PageShape shape, int pieces, int groups) {
  const nvfp4_kv_cache& c = caches.shape;
  const int rest = blockIdx.x / groups, p = blockIdx.x % groups * kCopyThreads + threadIdx.x;
  const int tensor = rest % (2 * caches.layers), i = rest / (2 * caches.layers);
  const int from = src[i], to = dst[i];
  if (from < 0 || from >= c.num_pages || to < 0 || to >= c.num_pages || from == to || p >= pieces) return;
  uint8_t* base = tensor % 2 ? caches.v[tensor / 2] : caches.k[tensor / 2];
  const int64_t page = c.page_stride * elem_size(c);
  int64_t at = (int64_t)p * 16;
  if (!WHOLE) {
    const int run = (int)(shape.run / 16), row = p / run, mid = (int)shape.mid;
    at = row / mid * shape.outer_stride + row % mid * shape.mid_stride + p % run * 16;
  }
  const u32x4_t held = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(base + from * page + at));
  __builtin_nontemporal_store(held, reinterpret_cast<u32x4_t*>(base + to * page + at));
}

hipError_t launch_kv_copy_pages(const int32_t* src, const int32_t* dst, int64_t n, const LayerCaches& caches,
                                hipStream_t stream) {
  const PageShape p = page_shape(caches.shape);
  const int pieces = (int)page_pieces(p), groups = (int)copy_groups(p);
  const dim3 grid((unsigned)(n * 2 * caches.layers * groups));
  if (p.mid == 1 && p.outer == 1)
    kv_copy_pages_kernel<true><<<grid, kCopyThreads, 0, stream>>>(src, dst, caches, p, pieces, groups);
  else
    kv_copy_pages_kernel<false><<<grid, kCopyThreads, 0, stream>>>(src, dst, caches, p, pieces, groups);
  return hipGetLastError();
}

}  // namespace nvfp4

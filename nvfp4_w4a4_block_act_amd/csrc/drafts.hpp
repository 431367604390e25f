// Host-side view of the operators that serve drafted tokens: the argument bundles that
// their launchers take, and the launchers.  The C ABI (api_drafts.cpp) sees only this
// header and launch.hpp, so it compiles as plain C++ against the HIP runtime API.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

struct TreeArgs {
  const uint16_t* q;
  int64_t ldq, ldt, ldo;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* parents;  // null: a chain
  nvfp4_kv_cache cache;
  uint16_t* out;
  float* lse;
  void* workspace;
  int B, nodes, q_heads, max_len, window;
  float scale;
};
size_t attn_tree_workspace(int64_t B, int nodes, int q_heads, int kv_heads, int head_dim, int64_t max_len, int64_t window);
hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t stream);

struct VerifyArgs {
  const float* logits;
  const float* draft;  // null: drafts picked without chance
  int64_t ld, ldd;
  const int64_t* drafts;
  const int32_t* parents;      // null: chains
  const float* temperature;    // null: greedy
  const float* uniforms;
  int64_t* tokens;
  int32_t* path;
  int32_t* counts;
  void* workspace;
  int B, nodes, vocab;
};
size_t verify_workspace(int64_t B, int nodes, int64_t vocab, bool sampled);
int64_t verify_groups(int64_t B, int nodes, int64_t vocab, bool sampled);  // workgroups of its largest launch
hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream);

// The caches of a model's layers, all of one shape.
struct LayerCaches {
  nvfp4_kv_cache shape;  // layer 0
  int layers;
  uint8_t* k[NVFP4_MAX_LAYERS];
  uint8_t* v[NVFP4_MAX_LAYERS];
};

struct CompactArgs {
  const int32_t* table;
  int64_t ldt;
  const int32_t* lens;
  const int32_t* path;
  const int32_t* counts;
  int B, nodes;
};
hipError_t launch_kv_compact(const CompactArgs& a, const LayerCaches& caches, hipStream_t stream);

// A page as nested runs of bytes: outer x mid runs of `run` contiguous ones.
struct PageShape {
  int64_t run, mid, mid_stride, outer, outer_stride;
};
PageShape page_shape(const nvfp4_kv_cache& c);
int64_t copy_groups(const PageShape& p);  // workgroups of one page of one tensor
hipError_t launch_kv_copy_pages(const int32_t* src, const int32_t* dst, int64_t n, const LayerCaches& caches,
                                hipStream_t stream);

}  // namespace nvfp4

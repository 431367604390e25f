// Host-side view of the token mixers: the argument bundles that their launchers
// take, and the launchers.  The C ABI (api_mixers.cpp) sees only this header and
// launch.hpp, so it compiles as plain C++ against the HIP runtime API.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t T, ldq, ldk, ldv, ldqo, max_pos;
  const float* rope;
  const int64_t* positions;
  const int64_t* slots;
  uint16_t* q_out;
  nvfp4_kv_cache cache;
  int q_heads, rot, interleaved, src_f32;
};
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream);

struct AttnArgs {
  const uint16_t* q;
  int64_t B, ldq, ldt, ldo;
  const int32_t* table;
  const int32_t* lens;
  nvfp4_kv_cache cache;
  uint16_t* out;
  float* lse;
  void* workspace;
  int q_heads, max_len, window;
  float scale;
};
size_t attn_decode_workspace(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t max_len, int64_t window);
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream);

struct GdnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* g;
  const float* beta;
  int64_t ldq, ldk, ldv, ldg, ldb, ldo;
  int64_t T, B, num_states;
  const int32_t* cu;         // prefill only
  const int32_t* has_state;  // prefill only
  const int32_t* index;
  float* state;
  uint16_t* out;
  void* workspace;
  int k_heads, v_heads, k_dim, v_dim;
  float scale;
};
hipError_t launch_gdn_step(const GdnArgs& a, hipStream_t stream);
size_t gdn_prefill_workspace(int64_t T, int64_t B, int k_heads, int v_heads, int k_dim, int v_dim);
hipError_t launch_gdn_prefill(const GdnArgs& a, hipStream_t stream);

}  // namespace nvfp4

// C ABI of the token mixers (paged cache append, decode attention, gated linear
// attention): argument validation and dispatch, by the same rules as api.cpp --
// everything is checked on the host before anything is enqueued, and this file
// compiles as plain C++ against the HIP runtime API.
#include <math.h>
#include <stdint.h>

#include "cache_checks.hpp"
#include "launch.hpp"
#include "mixers.hpp"

namespace {

using namespace nvfp4::checks;

nvfp4_status check_append(const nvfp4::AppendArgs& a, int32_t src_dtype, const nvfp4_kv_cache* cache) {
  const nvfp4_status s = check_cache(cache);
  if (s != NVFP4_OK) return s;
  if (a.T < 0 || a.max_pos < 0 || (src_dtype != NVFP4_F32 && src_dtype != NVFP4_BF16)) return NVFP4_EINVAL;
  if (a.q ? (a.q_heads < 1 || !a.q_out) : a.q_out != nullptr) return NVFP4_EINVAL;
  const int64_t dim = cache->head_dim, kv = cache->kv_heads * dim, qw = a.q ? a.q_heads * dim : 0;
  if (a.rot < 0 || a.rot > dim || a.rot % 16 != 0 || a.T >= kMaxDim || a.max_pos >= kMaxDim || a.q_heads > kMaxHeads)
    return NVFP4_ESHAPE;
  if (!ld_ok(a.ldk, kv) || !ld_ok(a.ldv, kv) || (a.q && (!ld_ok(a.ldq, qw) || !ld_ok(a.ldqo, qw)))) return NVFP4_ESHAPE;
  if (a.T > kMaxGroups) return NVFP4_ESHAPE;
  if (a.T == 0) return NVFP4_OK;
  if (!a.k || !a.v || !a.slots || (a.rot > 0 && (!a.rope || !a.positions))) return NVFP4_EINVAL;
  const int elem = src_dtype == NVFP4_F32 ? 4 : 2, unit = 16 / elem;
  if (!all_aligned({a.q, a.k, a.v, a.rope, a.positions, a.slots, a.q_out, a.q_norm, a.k_norm})) return NVFP4_EALIGN;
  if (a.ldk % unit || a.ldv % unit || (a.q && (a.ldq % unit || a.ldqo % 8))) return NVFP4_EALIGN;
  const size_t span = (size_t)cache_span(*cache) * cache_elem(*cache);
  const Buf ins[] = {{a.q, extent(a.T, qw, a.ldq, elem)},
                     {a.k, extent(a.T, kv, a.ldk, elem)},
                     {a.v, extent(a.T, kv, a.ldv, elem)},
                     {a.rope, a.rot ? (size_t)(a.max_pos * a.rot) * 4 : 0},
                     {a.positions, a.rot ? (size_t)a.T * 8 : 0},
                     {a.slots, (size_t)a.T * 8},
                     {a.q_norm, (size_t)dim * 4},
                     {a.k_norm, (size_t)dim * 4},
                     {cache->k_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u},
                     {cache->v_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u}};
  // k and v of the cache may lie interleaved: check_cache holds their rows against each other
  const Buf k_outs[] = {{cache->k, span}, {a.q_out, extent(a.T, qw, a.ldqo, 2)}};
  const Buf v_outs[] = {{cache->v, span}, {a.q_out, extent(a.T, qw, a.ldqo, 2)}};
  return disjoint(k_outs, ins) && disjoint(v_outs, ins) ? NVFP4_OK : NVFP4_EINVAL;
}

nvfp4_status check_attn(const nvfp4::AttnArgs& a, const nvfp4_kv_cache* cache, int64_t max_len, int64_t window,
                        size_t workspace_bytes) {
  const nvfp4_status s = check_cache(cache);
  if (s != NVFP4_OK) return s;
  if (a.B < 0 || a.q_heads < 1 || max_len < 0 || window < 0 || !isfinite(a.scale)) return NVFP4_EINVAL;
  const int64_t width = (int64_t)a.q_heads * cache->head_dim;
  if (a.q_heads % cache->kv_heads != 0 || a.q_heads > kMaxHeads || a.B >= kMaxDim || max_len > kMaxLen ||
      window >= kMaxDim || !ld_ok(a.ldq, width) || !ld_ok(a.ldo, width) || a.ldt < 0 || a.ldt >= kMaxDim ||
      a.ldt < (max_len + cache->page_size - 1) / cache->page_size)
    return NVFP4_ESHAPE;
  if (a.B > 65535 || (a.B + 7) * a.q_heads > kMaxGroups) return NVFP4_ESHAPE;
  if (a.B == 0) return NVFP4_OK;
  if (!a.q || !a.out || !a.lens || (max_len > 0 && !a.table)) return NVFP4_EINVAL;
  if (!all_aligned({a.q, a.out, a.lse, a.lens, a.table})) return NVFP4_EALIGN;
  if (a.ldq % 8 || a.ldo % 8) return NVFP4_EALIGN;
  const size_t need =
      nvfp4::attn_decode_workspace(a.B, a.q_heads, cache->kv_heads, cache->head_dim, max_len, window);
  if (need > 0 && (!a.workspace || workspace_bytes < need)) return NVFP4_EWORKSPACE;
  if (need > 0 && !aligned16(a.workspace)) return NVFP4_EALIGN;
  const size_t span = (size_t)cache_span(*cache) * cache_elem(*cache);
  const Buf outs[] = {{a.out, extent(a.B, width, a.ldo, 2)},
                      {a.lse, (size_t)(a.B * a.q_heads) * 4},
                      {a.workspace, need}};
  const Buf ins[] = {{a.q, extent(a.B, width, a.ldq, 2)},
                     {cache->k, span},
                     {cache->v, span},
                     {a.lens, (size_t)a.B * 4},
                     {a.table, max_len ? (size_t)(a.B * a.ldt) * 4 : 0},
                     {cache->k_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u},
                     {cache->v_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u}};
  return disjoint(outs, ins) ? NVFP4_OK : NVFP4_EINVAL;
}

// The recurrent layer's arguments; `rows` tokens, `prefill` with the sequence table.
nvfp4_status check_gdn(const nvfp4::GdnArgs& a, bool prefill, size_t workspace_bytes) {
  const int64_t rows = prefill ? a.T : a.B;
  if (a.B < 0 || a.T < 0 || a.k_heads < 1 || a.v_heads < 1 || a.num_states < 0 || !isfinite(a.scale))
    return NVFP4_EINVAL;
  if ((a.k_dim != 64 && a.k_dim != 128) || a.v_dim < 32 || a.v_dim > 1024 || a.v_dim % 32 != 0) return NVFP4_ESHAPE;
  if (a.v_heads % a.k_heads != 0 || a.v_heads > 65535 || rows >= kMaxDim || a.B > 65535 || a.num_states >= kMaxDim)
    return NVFP4_ESHAPE;
  if ((a.B * a.v_heads + 7) * (a.v_dim / 16) > kMaxGroups) return NVFP4_ESHAPE;
  if (prefill && (a.T / 64 + a.B + 8) * (a.v_heads / a.k_heads) > kMaxGroups) return NVFP4_ESHAPE;
  if (!a.index && a.num_states < a.B) return NVFP4_ESHAPE;
  const int64_t kw = (int64_t)a.k_heads * a.k_dim, vw = (int64_t)a.v_heads * a.v_dim;
  if (!ld_ok(a.ldq, kw) || !ld_ok(a.ldk, kw) || !ld_ok(a.ldv, vw) || !ld_ok(a.ldo, vw) || !ld_ok(a.ldg, a.v_heads) ||
      (a.beta && !ld_ok(a.ldb, a.v_heads)))
    return NVFP4_ESHAPE;
  const int64_t each = vw * a.k_dim;  // at most 2^33
  if (a.num_states > 0 && each > ((int64_t)1 << 58) / a.num_states) return NVFP4_ESHAPE;
  if (a.B == 0) return NVFP4_OK;
  if (a.num_states > 0 && !a.state) return NVFP4_EINVAL;
  if (prefill && !a.cu) return NVFP4_EINVAL;
  if (rows > 0 && (!a.q || !a.k || !a.v || !a.g || !a.out)) return NVFP4_EINVAL;
  if (!all_aligned({a.q, a.k, a.v, a.state, a.index, a.cu, a.has_state, a.out})) return NVFP4_EALIGN;
  // gates are read one value at a time, from column ranges of any width
  if (((reinterpret_cast<uintptr_t>(a.g) | reinterpret_cast<uintptr_t>(a.beta)) & 3u) != 0) return NVFP4_EALIGN;
  if (a.ldq % 8 || a.ldk % 8 || a.ldv % 8 || a.ldo % 8) return NVFP4_EALIGN;
  const size_t need =
      prefill ? nvfp4::gdn_prefill_workspace(a.T, a.B, a.k_heads, a.v_heads, a.k_dim, a.v_dim) : 0;
  if (need > 0 && (!a.workspace || workspace_bytes < need)) return NVFP4_EWORKSPACE;
  if (need > 0 && !aligned16(a.workspace)) return NVFP4_EALIGN;
  const Buf outs[] = {{a.state, (size_t)(a.num_states * each) * 4}, {a.out, extent(rows, vw, a.ldo, 2)},
                      {a.workspace, need}};
  const Buf ins[] = {{a.q, extent(rows, kw, a.ldq, 2)},
                     {a.k, extent(rows, kw, a.ldk, 2)},
                     {a.v, extent(rows, vw, a.ldv, 2)},
                     {a.g, extent(rows, a.v_heads, a.ldg, 4)},
                     {a.beta, extent(rows, a.v_heads, a.ldb, 4)},
                     {a.index, (size_t)a.B * 4},
                     {a.cu, prefill ? (size_t)(a.B + 1) * 4 : 0},
                     {a.has_state, prefill ? (size_t)a.B * 4 : 0}};
  return disjoint(outs, ins) ? NVFP4_OK : NVFP4_EINVAL;
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_append(const void* q, const void* k, const void* v, int32_t src_dtype, int64_t T,
                             int32_t q_heads, int64_t ldq, int64_t ldk, int64_t ldv, const float* rope,
                             int32_t rot_dim, int64_t max_pos, int32_t interleaved, const int64_t* positions,
                             const int64_t* slots, const nvfp4_kv_cache* cache, void* q_out, int64_t ldqo,
                             void* stream) {
  nvfp4::AppendArgs a{q,     k,         v,     T, ldq, ldk, ldv, ldqo, max_pos, rope, positions, slots,
                      static_cast<uint16_t*>(q_out), {}, q_heads, rot_dim, interleaved != 0, src_dtype == NVFP4_F32};
  const nvfp4_status s = check_append(a, src_dtype, cache);
  if (s != NVFP4_OK || T == 0) return s;
  a.cache = *cache;
  return launched(nvfp4::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_append_norm(const void* q, const void* k, const void* v, int32_t src_dtype, int64_t T,
                                  int32_t q_heads, int64_t ldq, int64_t ldk, int64_t ldv, const float* q_norm,
                                  const float* k_norm, float eps, const float* rope, int32_t rot_dim, int64_t max_pos,
                                  int32_t interleaved, const int64_t* positions, const int64_t* slots,
                                  const nvfp4_kv_cache* cache, void* q_out, int64_t ldqo, void* stream) {
  nvfp4::AppendArgs a{q,     k,         v,     T, ldq, ldk, ldv, ldqo, max_pos, rope, positions, slots,
                      static_cast<uint16_t*>(q_out), {}, q_heads, rot_dim, interleaved != 0, src_dtype == NVFP4_F32,
                      q_norm, k_norm, eps};
  if (!isfinite(eps) || eps < 0.0f || (q_norm && !q && T > 0)) return NVFP4_EINVAL;
  const nvfp4_status s = check_append(a, src_dtype, cache);
  if (s != NVFP4_OK || T == 0) return s;
  a.cache = *cache;
  return launched(nvfp4::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_attn_decode_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t max_len, int64_t window) {
  if (B < 1 || B > 65535 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || q_heads > kMaxHeads ||
      head_dim < 1 || head_dim > 256 || max_len < 0 || window < 0 || max_len > kMaxLen || window >= kMaxDim)
    return 0;
  return nvfp4::attn_decode_workspace(B, q_heads, kv_heads, head_dim, max_len, window);
}

nvfp4_status nvfp4_attn_decode(const void* q_bf16, int64_t B, int32_t q_heads, int64_t ldq,
                               const nvfp4_kv_cache* cache, const int32_t* block_table, int64_t ldt,
                               const int32_t* seq_lens, int64_t max_len, float scale, int64_t window,
                               void* out_bf16, int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream) {
  nvfp4::AttnArgs a{u16(q_bf16), B, ldq, ldt, ldo, block_table, seq_lens, {}, static_cast<uint16_t*>(out_bf16), lse,
                    workspace, q_heads, 0, 0, scale};
  const nvfp4_status s = check_attn(a, cache, max_len, window, workspace_bytes);
  if (s != NVFP4_OK || B == 0) return s;
  a.cache = *cache;
  a.max_len = (int)max_len;
  a.window = (int)window;
  return launched(nvfp4::launch_attn_decode(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_gdn_step(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                            const float* g, int64_t ldg, const float* beta, int64_t ldb, int64_t B, int32_t k_heads,
                            int32_t v_heads, int32_t k_dim, int32_t v_dim, float* state, int64_t num_states,
                            const int32_t* state_index, float scale, void* out, int64_t ldo, void* stream) {
  const nvfp4::GdnArgs a{u16(q), u16(k), u16(v), g,     beta,    ldq,     ldk,   ldv,   ldg,
                         ldb,    ldo,    B,      B,     num_states, nullptr, nullptr, state_index, state,
                         static_cast<uint16_t*>(out), nullptr, k_heads, v_heads, k_dim, v_dim, scale};
  const nvfp4_status s = check_gdn(a, false, 0);
  if (s != NVFP4_OK || B == 0) return s;
  return launched(nvfp4::launch_gdn_step(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_gdn_prefill_workspace_bytes(int64_t T, int64_t B, int32_t k_heads, int32_t v_heads, int32_t k_dim,
                                         int32_t v_dim) {
  if (T < 0 || T >= kMaxDim || B < 1 || B > 65535 || k_heads < 1 || v_heads < 1 || v_heads > 65535 || k_dim < 1 ||
      k_dim > 128 || v_dim < 1 || v_dim > 1024)
    return 0;
  return nvfp4::gdn_prefill_workspace(T, B, k_heads, v_heads, k_dim, v_dim);
}

nvfp4_status nvfp4_gdn_prefill(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const float* g, int64_t ldg, const float* beta, int64_t ldb, int64_t T, int64_t B,
                               const int32_t* cu_seqlens, int32_t k_heads, int32_t v_heads, int32_t k_dim,
                               int32_t v_dim, float* state, int64_t num_states, const int32_t* state_index,
                               const int32_t* has_state, float scale, void* out, int64_t ldo, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const nvfp4::GdnArgs a{u16(q), u16(k), u16(v), g,     beta,    ldq,     ldk,   ldv,   ldg,
                         ldb,    ldo,    T,      B,     num_states, cu_seqlens, has_state, state_index, state,
                         static_cast<uint16_t*>(out), workspace, k_heads, v_heads, k_dim, v_dim, scale};
  const nvfp4_status s = check_gdn(a, true, workspace_bytes);
  if (s != NVFP4_OK || B == 0) return s;
  return launched(nvfp4::launch_gdn_prefill(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// C ABI of the operators that serve drafted tokens (tree attention, verification, cache rows
// and pages that move): argument validation and dispatch, by the same rules as api.cpp --
// everything is checked on the host before anything is enqueued, and this file compiles as
// plain C++ against the HIP runtime API.
#include <math.h>
#include <stdint.h>

#include "cache_checks.hpp"
#include "drafts.hpp"
#include "launch.hpp"

namespace {

using namespace nvfp4::checks;

constexpr int kMaxNodes = NVFP4_MAX_NODES;
constexpr int64_t kMaxCopies = (1 << 24) - 1;  // workgroups of 256 threads: below 2^32 threads

nvfp4_status check_tree(const nvfp4::TreeArgs& a, int64_t B, const nvfp4_kv_cache* cache, int64_t max_len, int64_t window,
                        size_t workspace_bytes) {
  const nvfp4_status s = check_cache(cache);
  if (s != NVFP4_OK) return s;
  if (B < 0 || a.nodes < 1 || a.q_heads < 1 || max_len < 0 || window < 0 || !isfinite(a.scale)) return NVFP4_EINVAL;
  const int64_t width = (int64_t)a.q_heads * cache->head_dim;
  if (a.nodes > kMaxNodes || a.q_heads % cache->kv_heads != 0 || a.q_heads > kMaxHeads || max_len > kMaxLen ||
      window >= kMaxDim || !ld_ok(a.ldq, width) || !ld_ok(a.ldo, width) || a.ldt < 0 || a.ldt >= kMaxDim ||
      a.ldt < (max_len + a.nodes + cache->page_size - 1) / cache->page_size)
    return NVFP4_ESHAPE;
  if (B > 65535 || (B + 7) * a.q_heads * a.nodes > kMaxGroups) return NVFP4_ESHAPE;
  if (B == 0) return NVFP4_OK;
  if (!a.q || !a.out || !a.lens || !a.table) return NVFP4_EINVAL;
  if (!all_aligned({a.q, a.out, a.lse, a.lens, a.table, a.parents})) return NVFP4_EALIGN;
  if (a.ldq % 8 || a.ldo % 8) return NVFP4_EALIGN;
  const size_t need =
      nvfp4::attn_tree_workspace(B, a.nodes, a.q_heads, cache->kv_heads, cache->head_dim, max_len, window);
  if (need > 0 && (!a.workspace || workspace_bytes < need)) return NVFP4_EWORKSPACE;
  if (need > 0 && !aligned16(a.workspace)) return NVFP4_EALIGN;
  const size_t span = (size_t)cache_span(*cache) * cache_elem(*cache);
  const int64_t rows = B * a.nodes;
  const Buf outs[] = {{a.out, extent(rows, width, a.ldo, 2)}, {a.lse, (size_t)(rows * a.q_heads) * 4}, {a.workspace, need}};
  const Buf ins[] = {{a.q, extent(rows, width, a.ldq, 2)},
                     {cache->k, span},
                     {cache->v, span},
                     {a.lens, (size_t)B * 4},
                     {a.table, (size_t)(B * a.ldt) * 4},
                     {a.parents, (size_t)rows * 4},
                     {cache->k_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u},
                     {cache->v_amax, cache->dtype == NVFP4_E4M3 ? 4u : 0u}};
  return disjoint(outs, ins) ? NVFP4_OK : NVFP4_EINVAL;
}

nvfp4_status check_verify(const nvfp4::VerifyArgs& a, int64_t B, int64_t vocab, size_t workspace_bytes) {
  if (B < 0 || a.nodes < 1 || vocab < 1) return NVFP4_EINVAL;
  if (a.nodes > kMaxNodes || B > 65535 || vocab > kMaxDim - 65536 || !ld_ok(a.ld, vocab) || (a.draft && !ld_ok(a.ldd, vocab)))
    return NVFP4_ESHAPE;
  if (nvfp4::verify_groups(B, a.nodes, vocab, a.draft != nullptr) > kMaxGroups) return NVFP4_ESHAPE;
  if (B == 0) return NVFP4_OK;
  if (!a.logits || !a.drafts || !a.tokens || !a.path || !a.counts || (a.temperature && !a.uniforms)) return NVFP4_EINVAL;
  if (!all_aligned({a.logits, a.draft, a.drafts, a.parents, a.temperature, a.uniforms, a.tokens, a.path, a.counts}))
    return NVFP4_EALIGN;
  const size_t need = nvfp4::verify_workspace(B, a.nodes, vocab, a.draft != nullptr);
  if (!a.workspace || workspace_bytes < need) return NVFP4_EWORKSPACE;
  if (!aligned16(a.workspace)) return NVFP4_EALIGN;
  const int64_t rows = B * a.nodes;
  const Buf outs[] = {{a.tokens, (size_t)rows * 8}, {a.path, (size_t)rows * 4}, {a.counts, (size_t)B * 4}, {a.workspace, need}};
  const Buf ins[] = {{a.logits, extent(rows, vocab, a.ld, 4)},
                     {a.draft, extent(rows, vocab, a.ldd, 4)},
                     {a.drafts, (size_t)rows * 8},
                     {a.parents, (size_t)rows * 4},
                     {a.temperature, (size_t)B * 4},
                     {a.uniforms, (size_t)(rows + B) * 4}};
  return disjoint(outs, ins) ? NVFP4_OK : NVFP4_EINVAL;
}

// The caches of all layers: one shape, no memory in common.
nvfp4_status check_layers(const nvfp4_kv_cache* caches, int32_t layers, nvfp4::LayerCaches& out) {
  if (!caches || layers < 1) return NVFP4_EINVAL;
  if (layers > NVFP4_MAX_LAYERS) return NVFP4_ESHAPE;
  for (int i = 0; i < layers; ++i) {
    const nvfp4_kv_cache &c = caches[i], &f = caches[0];
    const nvfp4_status s = check_cache(&c);
    if (s != NVFP4_OK) return s;
    if (c.num_pages != f.num_pages || c.page_stride != f.page_stride || c.token_stride != f.token_stride ||
        c.head_stride != f.head_stride || c.page_size != f.page_size || c.kv_heads != f.kv_heads ||
        c.head_dim != f.head_dim || c.dtype != f.dtype)
      return NVFP4_ESHAPE;
    out.k[i] = static_cast<uint8_t*>(c.k), out.v[i] = static_cast<uint8_t*>(c.v);
  }
  out.shape = caches[0];
  out.layers = layers;
  const Axes axes = axes_of(out.shape);
  const size_t span = (size_t)cache_span(out.shape) * cache_elem(out.shape);
  auto apart = [&](const uint8_t* x, const uint8_t* y) {
    return !overlap({x, span}, {y, span}) || bases_disjoint(out.shape, axes, x, y);
  };
  for (int i = 0; i < layers; ++i)
    for (int j = i + 1; j < layers; ++j)
      if (!apart(out.k[i], out.k[j]) || !apart(out.k[i], out.v[j]) || !apart(out.v[i], out.k[j]) || !apart(out.v[i], out.v[j]))
        return NVFP4_EINVAL;
  return NVFP4_OK;
}

// No row of a cache overlaps a buffer that the call reads.
template <int N>
bool clear_of(const nvfp4::LayerCaches& c, const Buf (&ins)[N]) {
  const size_t span = (size_t)cache_span(c.shape) * cache_elem(c.shape);
  for (int i = 0; i < c.layers; ++i)
    for (const Buf& b : ins)
      if (overlap({c.k[i], span}, b) || overlap({c.v[i], span}, b)) return false;
  return true;
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

size_t nvfp4_attn_tree_workspace_bytes(int64_t B, int32_t nodes, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                       int64_t max_len, int64_t window) {
  if (B < 1 || B > 65535 || nodes < 1 || nodes > kMaxNodes || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 ||
      q_heads > kMaxHeads || head_dim < 1 || head_dim > 256 || max_len < 0 || window < 0 || max_len > kMaxLen ||
      window >= kMaxDim || (B + 7) * q_heads * nodes > kMaxGroups)
    return 0;
  return nvfp4::attn_tree_workspace(B, nodes, q_heads, kv_heads, head_dim, max_len, window);
}

nvfp4_status nvfp4_attn_tree(const void* q_bf16, int64_t B, int32_t nodes, int32_t q_heads, int64_t ldq,
                             const nvfp4_kv_cache* cache, const int32_t* block_table, int64_t ldt, const int32_t* ctx_lens,
                             const int32_t* parents, int64_t max_len, float scale, int64_t window, void* out_bf16,
                             int64_t ldo, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4::TreeArgs a{u16(q_bf16), ldq, ldt, ldo, block_table, ctx_lens, parents, {}, static_cast<uint16_t*>(out_bf16), lse,
                    workspace, 0, nodes, q_heads, 0, 0, scale};
  const nvfp4_status s = check_tree(a, B, cache, max_len, window, workspace_bytes);
  if (s != NVFP4_OK || B == 0) return s;
  a.cache = *cache;
  a.B = (int)B;
  a.max_len = (int)max_len;
  a.window = (int)window;
  return launched(nvfp4::launch_attn_tree(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_verify_drafts_workspace_bytes(int64_t B, int32_t nodes, int64_t vocab, int32_t with_draft_logits) {
  if (B < 1 || B > 65535 || nodes < 1 || nodes > kMaxNodes || vocab < 1 || vocab > kMaxDim - 65536) return 0;
  return nvfp4::verify_workspace(B, nodes, vocab, with_draft_logits != 0);
}

nvfp4_status nvfp4_verify_drafts(const float* logits, int64_t B, int32_t nodes, int64_t vocab, int64_t ld,
                                 const float* draft_logits, int64_t ldd, const int64_t* drafts, const int32_t* parents,
                                 const float* temperature, const float* uniforms, int64_t* tokens, int32_t* path,
                                 int32_t* counts, void* workspace, size_t workspace_bytes, void* stream) {
  // the greedy rule asks no draft model
  nvfp4::VerifyArgs a{logits, temperature ? draft_logits : nullptr, ld, ldd, drafts, parents, temperature, uniforms, tokens,
                      path, counts, workspace, 0, nodes, 0};
  const nvfp4_status s = check_verify(a, B, vocab, workspace_bytes);
  if (s != NVFP4_OK || B == 0) return s;
  a.B = (int)B;
  a.vocab = (int)vocab;
  return launched(nvfp4::launch_verify(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_compact(const nvfp4_kv_cache* caches, int32_t layers, const int32_t* block_table, int64_t ldt,
                              int64_t B, int32_t nodes, const int32_t* ctx_lens, const int32_t* path,
                              const int32_t* counts, void* stream) {
  nvfp4::LayerCaches c{};
  const nvfp4_status s = check_layers(caches, layers, c);
  if (s != NVFP4_OK) return s;
  if (B < 0 || nodes < 1 || ldt < 0) return NVFP4_EINVAL;
  if (nodes > kMaxNodes || B > 65535 || ldt >= kMaxDim || B * layers * 2 * c.shape.kv_heads > kMaxGroups) return NVFP4_ESHAPE;
  if (B == 0) return NVFP4_OK;
  if (!ctx_lens || !path || !counts || (ldt > 0 && !block_table)) return NVFP4_EINVAL;
  if (!all_aligned({block_table, ctx_lens, path, counts})) return NVFP4_EALIGN;
  const Buf ins[] = {{block_table, (size_t)(B * ldt) * 4},
                     {ctx_lens, (size_t)B * 4},
                     {path, (size_t)(B * nodes) * 4},
                     {counts, (size_t)B * 4}};
  if (!clear_of(c, ins)) return NVFP4_EINVAL;
  return launched(nvfp4::launch_kv_compact({block_table, ldt, ctx_lens, path, counts, (int)B, nodes}, c,
                                           static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_copy_pages(const nvfp4_kv_cache* caches, int32_t layers, const int32_t* src, const int32_t* dst,
                                 int64_t n, void* stream) {
  nvfp4::LayerCaches c{};
  const nvfp4_status s = check_layers(caches, layers, c);
  if (s != NVFP4_OK) return s;
  if (n < 0) return NVFP4_EINVAL;
  const int64_t groups = nvfp4::copy_groups(nvfp4::page_shape(c.shape));
  if (n >= kMaxDim || n > kMaxCopies / (2 * layers * groups)) return NVFP4_ESHAPE;
  if (n == 0) return NVFP4_OK;
  if (!src || !dst) return NVFP4_EINVAL;
  if (!all_aligned({src, dst})) return NVFP4_EALIGN;
  const Buf ins[] = {{src, (size_t)n * 4}, {dst, (size_t)n * 4}};
  if (!clear_of(c, ins)) return NVFP4_EINVAL;
  return launched(nvfp4::launch_kv_copy_pages(src, dst, n, c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

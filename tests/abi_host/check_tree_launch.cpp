// Host-only check of the tree attention's launches (attn_tree.hip), recorded by
// launch_recorder.hpp, and of how it splits sequences.  Prints one line per failed case and
// "ok <n>" at the end.
#include "launch_recorder.hpp"

#include <cstdint>
#include <cstdio>

#include "../../nvfp4_w4a4_block_act_amd/csrc/drafts.hpp"
#include "../../nvfp4_w4a4_block_act_amd/csrc/tree_splits.hpp"

namespace {
int bad = 0, n = 0;

nvfp4::TreeArgs args(int B, int nodes, int kv, int group, int dim, bool fp8, int max_len, int window) {
  nvfp4::TreeArgs a{};
  a.B = B, a.nodes = nodes, a.q_heads = kv * group, a.max_len = max_len, a.window = window, a.scale = 1.0f;
  a.cache.kv_heads = kv, a.cache.head_dim = dim, a.cache.dtype = fp8 ? NVFP4_E4M3 : NVFP4_BF16;
  a.cache.page_size = 16;
  return a;
}
}  // namespace

int main() {
  // One bound of dynamic LDS for each kernel, whatever the call, and every launch inside it and
  // inside a CU's LDS; a rejected launch ends the call.
  std::map<std::string, int> bound;
  for (int dim : {64, 128, 256})
    for (int fp8 : {0, 1})
      for (int nodes : {1, 2, 5, 16, 33, 64})
        for (int group : {1, 3, 5, 16, 24})
          for (int B : {1, 40})
            for (int max_len : {0, 700, 5000, 100000}) {
              const nvfp4::TreeArgs a = args(B, nodes, 2, group, dim, fp8, max_len, max_len == 5000 ? 3000 : 0);
              launches.clear();
              bounds_set.clear();
              if (nvfp4::launch_attn_tree(a, nullptr) != hipSuccess) ++bad;
              for (const auto& s : bounds_set) {
                if (bound.count(s.first) && bound[s.first] != s.second) printf("%s: two bounds\n", s.first.c_str()), ++bad;
                bound[s.first] = s.second;
              }
              for (const Launch& l : launches)
                if ((l.lds > 48 * 1024 && l.lds > l.lds_bound) || l.lds > 160 * 1024 - 4096 || l.grid.x > (1u << 22) || l.block.x > 1024)
                  printf("%s: %zu bytes of LDS, bound %zu, grid %u\n", l.kernel.c_str(), l.lds, l.lds_bound, l.grid.x), ++bad;
              const size_t all = launches.size();
              const bool split = nvfp4::attn_tree_workspace(B, nodes, 2 * group, 2, dim, max_len, a.window) > 0;
              if (all != (split ? 2u : 1u)) printf("%zu launches, splits %d\n", all, split), ++bad;
              for (size_t i = 0; i < all; ++i) {
                launches.clear();
                fail_launch = (int)i;
                if (nvfp4::launch_attn_tree(a, nullptr) == hipSuccess || launches.size() != i)
                  printf("launch %zu of %zu rejected, but the call goes on\n", i, all), ++bad;
              }
              fail_launch = -1;
              ++n;
            }
  // A sequence of any length under the bound has no more splits than the launch, all of whole tiles.
  for (int64_t rows : {1, 7, 72, 100, 384, 2000, 100000})
    for (int64_t max_len : {0, 1, 31, 500, 1024, 4099, 33333, 1 << 20, 1 << 30})
      for (int64_t window : {0, 1, 100, 5000})
        for (int nodes : {1, 17, 64}) {
          const nvfp4::Splits s = nvfp4::tree_splits(rows, max_len, nodes, window);
          const int64_t span_bound = nvfp4::tree_span(max_len, nodes, window);
          if (s.count < 1 || s.tokens % nvfp4::kTreeTile || (int64_t)s.count * s.tokens < span_bound)
            printf("splits %d of %d for %lld\n", s.count, s.tokens, (long long)span_bound), ++bad;
          for (int64_t len = 0; len <= max_len; len = len * 3 / 2 + 1) {
            const int64_t begin = window > 0 && window < len ? (len - window) / nvfp4::kTreeTile * nvfp4::kTreeTile : 0;
            const int64_t span = len + nodes - begin;
            if (span > span_bound) printf("span %lld above %lld\n", (long long)span, (long long)span_bound), ++bad;
            const int t = s.count == 1 ? s.tokens : nvfp4::tree_split_tokens((int)rows, s.tokens, (int)span_bound, (int)span);
            if (t < nvfp4::kTreeTile || t % nvfp4::kTreeTile || (span + t - 1) / t > s.count)
              printf("rows %lld, %lld of %lld: %d splits of %d, sequence's %d\n", (long long)rows, (long long)span, (long long)span_bound,
                     s.count, s.tokens, t), ++bad;
            ++n;
          }
        }
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

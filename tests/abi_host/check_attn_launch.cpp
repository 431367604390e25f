// Host-only check of the decode attention's launches (attn_decode.hip), recorded by
// launch_recorder.hpp.  Prints one line per failed case and "ok <n>" at the end.
#include "launch_recorder.hpp"

#include <cstdint>
#include <cstdio>

#include "../../nvfp4_w4a4_block_act_amd/csrc/mixers.hpp"

namespace {
int bad = 0, n = 0;

nvfp4::AttnArgs args(int64_t B, int kv, int group, int dim, bool fp8, int max_len, int window) {
  nvfp4::AttnArgs a{};
  a.B = B, a.q_heads = kv * group, a.max_len = max_len, a.window = window, a.scale = 1.0f;
  a.cache.kv_heads = kv, a.cache.head_dim = dim, a.cache.dtype = fp8 ? NVFP4_E4M3 : NVFP4_BF16;
  a.cache.page_size = 16;
  return a;
}
}  // namespace

int main() {
  // A kernel's bound of dynamic LDS is set for the whole process: were it the size of the call
  // at hand, a call with fewer heads in another thread could lower it between the setting and
  // the launch.  So one kernel gets one size, and that holds every launch.
  std::map<std::string, int> bound;
  for (int dim : {64, 128, 256})
    for (int fp8 : {0, 1})
      for (int group = 1; group <= 33; ++group)
        for (int64_t B : {1, 64, 300})
          for (int max_len : {1, 700, 5000}) {
            launches.clear();
            bounds_set.clear();
            if (nvfp4::launch_attn_decode(args(B, 2, group, dim, fp8, max_len, 0), nullptr) != hipSuccess) ++bad;
            for (const auto& s : bounds_set) {
              if (bound.count(s.first) && bound[s.first] != s.second) {
                if (bad++ < 10)
                  printf("%s: bound set to %d after %d (group %d)\n", s.first.c_str(), s.second, bound[s.first], group);
              }
              bound[s.first] = s.second;
            }
            for (const Launch& l : launches)
              if (l.lds > 48 * 1024 && l.lds > l.lds_bound) {
                printf("%s: %zu bytes of LDS under a bound of %zu\n", l.kernel.c_str(), l.lds, l.lds_bound);
                ++bad;
              }
            const size_t all = launches.size();
            if (all == 0) ++bad;
            for (size_t i = 0; i < all; ++i) {  // whichever launch is rejected, the call says so and launches no more
              launches.clear();
              fail_launch = (int)i;
              if (nvfp4::launch_attn_decode(args(B, 2, group, dim, fp8, max_len, 0), nullptr) == hipSuccess ||
                  launches.size() != i)
                printf("launch %zu of %zu rejected, but the call goes on\n", i, all), ++bad;
            }
            fail_launch = -1;
            ++n;
          }
  if (bound.empty()) printf("no bound was set\n"), ++bad;
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

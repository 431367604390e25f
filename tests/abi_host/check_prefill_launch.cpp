// Host-only check of the gated delta rule prompts' launches (gdn_prefill.hip), recorded by
// launch_recorder.hpp: what each form launches, grids within a launch's limits at the ends of
// the sizes' ranges, and whichever launch is rejected, the call says so and launches no more.
// Prints one line per failed case and "ok <n>" at the end.
#include "launch_recorder.hpp"

#include <cstdint>
#include <cstdio>

#include "../../nvfp4_w4a4_block_act_amd/csrc/mixers.hpp"

namespace {
int bad = 0, n = 0;

nvfp4::GdnArgs args(int64_t T, int64_t B, int hk, int hv, int dk, int dv, bool delta) {
  static float beta;
  nvfp4::GdnArgs a{};
  a.T = T, a.B = B, a.num_states = B, a.k_heads = hk, a.v_heads = hv, a.k_dim = dk, a.v_dim = dv;
  a.beta = delta ? &beta : nullptr;
  return a;
}
bool has(const Launch& l, const char* part) { return l.kernel.find(part) != std::string::npos; }

void check(const nvfp4::GdnArgs& a, std::vector<const char*> want) {
  launches.clear();
  fail_launch = -1;
  const hipError_t e = nvfp4::launch_gdn_prefill(a, nullptr);
  bool ok = e == hipSuccess && launches.size() == want.size();
  for (size_t i = 0; ok && i < want.size(); ++i) ok = has(launches[i], want[i]);
  for (const Launch& l : launches)
    ok = ok && l.grid.x > 0 && l.grid.y > 0 && l.grid.y <= 65535 && (uint64_t)l.grid.x * l.block.x < (1ull << 32);
  if (!ok) {
    printf("T %ld B %ld heads %d/%d dims %d x %d:", (long)a.T, (long)a.B, a.k_heads, a.v_heads, a.k_dim, a.v_dim);
    for (const Launch& l : launches) printf(" %s (%u, %u)", l.kernel.c_str(), l.grid.x, l.grid.y);
    printf("\n");
    ++bad;
  }
  for (size_t i = 0; i < want.size(); ++i) {
    launches.clear();
    fail_launch = (int)i;
    if (nvfp4::launch_gdn_prefill(a, nullptr) == hipSuccess || launches.size() != i) {
      printf("launch %zu of %s rejected, but the call goes on\n", i, want[i]);
      ++bad;
    }
  }
  fail_launch = -1;
  ++n;
}
}  // namespace

int main() {
  for (bool delta : {true, false}) {
    // the template arguments: key dimension, tiles of 16 columns, delta rule
    check(args(8192, 1, 16, 32, 128, 128, delta), {"gdn_chunk_kernelILi128E", "gdn_state_kernelILi128ELi1E"});
    check(args(8192, 2, 16, 32, 128, 128, delta), {"gdn_chunk_kernelILi128E", "gdn_state_kernelILi128ELi2E"});
    check(args(8192, 4, 16, 32, 64, 128, delta),
          {"gdn_chunk_kernelILi64E", delta ? "gdn_state_kernelILi64ELi2E" : "gdn_state_kernelILi64ELi4E"});
    // whole heads: long sequences by columns before, where there is room for one
    check(args(8000, 8, 16, 32, 128, 128, delta), {"gdn_chunk_kernel", "gdn_state_kernelILi128ELi2E", "gdn_head_kernelILi128E"});
    check(args(100, 300, 64, 256, 64, 128, delta), {"gdn_chunk_kernel", "gdn_head_kernelILi64E"});
    check(args(0, 3, 2, 4, 128, 64, delta), {"gdn_state_kernel"});
    check(args(0, 300, 2, 4, 128, 128, delta), {"gdn_state_kernel", "gdn_head_kernel"});
    // the largest calls that the argument checks let pass
    check(args(((int64_t)1 << 28) - 1024, 1, 1, 1, 128, 32, delta), {"gdn_chunk_kernel", "gdn_state_kernel"});
    check(args(64, 65535, 1, 1, 128, 1024, delta), {"gdn_chunk_kernel", "gdn_state_kernel", "gdn_head_kernel"});
    check(args(64, 1, 65535, 65535, 64, 1024, delta), {"gdn_chunk_kernel", "gdn_head_kernel"});
  }
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

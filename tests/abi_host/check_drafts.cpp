// Host-only check of the argument handling for drafted tokens (api_drafts.cpp), built with the
// address and undefined-behaviour sanitizers against stand-in launchers: rejected calls request
// no launch, accepted ones one, and a launch the runtime rejects comes back as NVFP4_EHIP.
// Buffers are fake device addresses, never dereferenced; sizes go to the ends of their
// ranges, so that an overflow in a check would show.
// Prints one line per failed case and "ok <n>" at the end.
#include <cstdint>
#include <cstdio>
#include <functional>
#include <limits>
#include <string>
#include <vector>

#include "../../nvfp4_w4a4_block_act_amd/csrc/drafts.hpp"

static int launches = 0;
static bool fail = false;
static hipError_t record() {
  ++launches;
  return fail ? hipErrorLaunchFailure : hipSuccess;
}
namespace nvfp4 {
size_t attn_tree_workspace(int64_t B, int nodes, int q_heads, int, int head_dim, int64_t max_len, int64_t) {
  return max_len >= 1024 ? (size_t)B * nodes * q_heads * head_dim * 4 : 0;
}
hipError_t launch_attn_tree(const TreeArgs&, hipStream_t) { return record(); }
size_t verify_workspace(int64_t B, int nodes, int64_t vocab, bool sampled) {
  return (size_t)B * nodes * (size_t)((vocab + 8191) / 8192) * (sampled ? 40 : 16);
}
int64_t verify_groups(int64_t B, int nodes, int64_t vocab, bool sampled) {
  return B * nodes * (sampled ? 2 : 1) * ((vocab + 8191) / 8192);
}
hipError_t launch_verify(const VerifyArgs&, hipStream_t) { return record(); }
hipError_t launch_kv_compact(const CompactArgs&, const LayerCaches&, hipStream_t) { return record(); }
PageShape page_shape(const nvfp4_kv_cache& c) { return {(int64_t)c.head_dim, c.kv_heads, c.head_stride, c.page_size, c.token_stride}; }
int64_t copy_groups(const PageShape& p) { return (p.run * p.mid * p.outer + 16383) / 16384; }
hipError_t launch_kv_copy_pages(const int32_t*, const int32_t*, int64_t, const LayerCaches&, hipStream_t) { return record(); }
}  // namespace nvfp4

namespace {
template <class T = void>
T* at(uintptr_t mb, uintptr_t off = 0) {
  return reinterpret_cast<T*>((uintptr_t(1) << 40) + (mb << 20) + off);
}
nvfp4_kv_cache cache() {
  return {at(0), at(64), nullptr, nullptr, 32, 16 * 1024, 1024, 128, 16, 8, 128, NVFP4_BF16};
}
nvfp4_status tree(const nvfp4_kv_cache& c, int64_t B = 4, int nodes = 8, int heads = 40, int64_t max_len = 500, int64_t ldt = 32,
                  int64_t window = 0, size_t wsb = 0, int64_t ld = 5120) {
  return nvfp4_attn_tree(at(128), B, nodes, heads, ld, &c, at<int32_t>(160), ldt, at<int32_t>(161), at<int32_t>(162), max_len, 0.5f,
                         window, at(192), ld, at<float>(224), at(256), wsb, nullptr);
}
nvfp4_status verify(int64_t B = 4, int nodes = 8, int64_t vocab = 32000, int64_t ld = 32000, bool drawn = false, int64_t ldd = 32000,
                    size_t wsb = 1 << 20) {
  return nvfp4_verify_drafts(at<float>(0), B, nodes, vocab, ld, drawn ? at<float>(200) : nullptr, ldd, at<int64_t>(64),
                             at<int32_t>(65), at<float>(66), at<float>(67), at<int64_t>(68), at<int32_t>(69), at<int32_t>(70),
                             at(71), wsb, nullptr);
}
nvfp4_status compact(const std::vector<nvfp4_kv_cache>& c, int32_t layers, int64_t B = 4, int nodes = 8, int64_t ldt = 32) {
  return nvfp4_kv_compact(c.data(), layers, at<int32_t>(160), ldt, B, nodes, at<int32_t>(161), at<int32_t>(162), at<int32_t>(163), nullptr);
}
nvfp4_status copy(const std::vector<nvfp4_kv_cache>& c, int32_t layers, int64_t n = 4) {
  return nvfp4_kv_copy_pages(c.data(), layers, at<int32_t>(160), at<int32_t>(161), n, nullptr);
}
struct Case {
  const char* name;
  std::function<nvfp4_status()> call;
  nvfp4_status want;
};
}  // namespace

int main() {
  const int64_t big = std::numeric_limits<int64_t>::max();
  const int32_t big32 = std::numeric_limits<int32_t>::max();
  auto with = [](auto set) {
    nvfp4_kv_cache c = cache();
    set(c);
    return c;
  };
  std::vector<nvfp4_kv_cache> many;
  for (int i = 0; i < 64; ++i) many.push_back(with([&](auto& c) { c.k = at(1000 + 2 * i), c.v = at(1001 + 2 * i); }));
  std::vector<nvfp4_kv_cache> wide;  // extents that overlap, rows that do not
  for (int i = 0; i < 64; ++i)
    wide.push_back(with([&](auto& c) { c.k = at(0, 2 * i * 32768), c.v = at(0, (2 * i + 1) * 32768), c.page_stride = 128 * 16384; }));
  std::vector<nvfp4_kv_cache> huge = {with([](auto& c) { c.num_pages = 1 << 16, c.page_stride = (1LL << 40) - 8, c.v = at(0, 2 * 16 * 1024); })};
  std::vector<nvfp4_kv_cache> none = {with([](auto& c) { c.num_pages = 0, c.k = c.v = nullptr; })};
  std::vector<nvfp4_kv_cache> rows = {with([](auto& c) { c.page_size = 1 << 20, c.token_stride = 1 << 12, c.page_stride = 1LL << 33, c.num_pages = 1, c.k = at(1 << 16), c.v = at(1 << 17); })};
  std::vector<Case> cases = {
      {"tree", [] { return tree(cache()); }, NVFP4_OK},
      {"tree empty pool", [=] { return tree(none[0]); }, NVFP4_OK},
      {"tree B max", [=] { return tree(cache(), big); }, NVFP4_ESHAPE},
      {"tree nodes max", [=] { return tree(cache(), 4, big32); }, NVFP4_ESHAPE},
      {"tree heads max", [] { return tree(cache(), 4, 8, 0x7FFFFFF8); }, NVFP4_ESHAPE},
      {"tree max_len max", [=] { return tree(cache(), 4, 8, 40, big, big); }, NVFP4_ESHAPE},
      {"tree max_len 2^30, nodes 64", [=] { return tree(cache(), 4, 64, 40, 1 << 30, (1 << 26) + 3); }, NVFP4_ESHAPE},
      {"tree window max", [=] { return tree(cache(), 4, 8, 40, 500, 32, big); }, NVFP4_ESHAPE},
      {"tree ld max", [=] { return tree(cache(), 4, 8, 40, 500, 32, 0, 0, big - 7); }, NVFP4_ESHAPE},
      {"tree launch too large", [] { return tree(cache(), 65535, 2); }, NVFP4_ESHAPE},
      {"tree workspace", [] { return tree(cache(), 4, 8, 40, 2000, 126, 0, 16); }, NVFP4_EWORKSPACE},
      {"verify", [] { return verify(); }, NVFP4_OK},
      {"verify drawn", [] { return verify(4, 8, 32000, 32000, true); }, NVFP4_OK},
      {"verify B max", [=] { return verify(big); }, NVFP4_ESHAPE},
      {"verify nodes max", [=] { return verify(4, big32); }, NVFP4_ESHAPE},
      {"verify vocab max", [=] { return verify(4, 8, big, big); }, NVFP4_ESHAPE},
      {"verify ld max", [=] { return verify(4, 8, 32000, big); }, NVFP4_ESHAPE},
      {"verify ldd max", [=] { return verify(4, 8, 32000, 32000, true, big); }, NVFP4_ESHAPE},
      {"verify launch too large", [] { return verify(65535, 64, 65536, 65536); }, NVFP4_ESHAPE},
      {"verify workspace", [] { return verify(4, 8, 32000, 32000, false, 0, 64); }, NVFP4_EWORKSPACE},
      {"compact", [=] { return compact(many, 64); }, NVFP4_OK},
      {"compact interleaved", [=] { return compact(wide, 64); }, NVFP4_OK},
      {"compact layers max", [=] { return compact(many, big32); }, NVFP4_ESHAPE},
      {"compact layers 0", [=] { return compact(many, 0); }, NVFP4_EINVAL},
      {"compact B max", [=] { return compact(many, 64, big); }, NVFP4_ESHAPE},
      {"compact nodes max", [=] { return compact(many, 64, 4, big32); }, NVFP4_ESHAPE},
      {"compact table max", [=] { return compact(many, 64, 4, 8, big); }, NVFP4_ESHAPE},
      {"compact widest pool", [=] { return compact(huge, 1); }, NVFP4_EINVAL},
      {"compact empty pool", [=] { return compact(none, 1); }, NVFP4_OK},
      {"compact launch too large", [=] { return compact(many, 64, 65535); }, NVFP4_ESHAPE},
      {"copy", [=] { return copy(many, 64); }, NVFP4_OK},
      {"copy interleaved", [=] { return copy(wide, 64); }, NVFP4_OK},
      {"copy n max", [=] { return copy(many, 1, big); }, NVFP4_ESHAPE},
      {"copy launch too large", [=] { return copy(many, 64, 1 << 20); }, NVFP4_ESHAPE},
      {"copy large pages", [=] { return copy(rows, 1, 1); }, NVFP4_OK},
      {"copy many large pages", [=] { return copy(rows, 1, 1 << 10); }, NVFP4_ESHAPE},
      {"copy empty pool", [=] { return copy(none, 1); }, NVFP4_OK},
  };
  int bad = 0, n = 0;
  for (const Case& c : cases) {
    launches = 0;
    fail = false;
    const nvfp4_status s = c.call();
    if (s != c.want || launches != (s == NVFP4_OK ? 1 : 0)) {
      printf("%s: status %d (want %d), %d launches\n", c.name, s, c.want, launches);
      ++bad;
    }
    if (c.want == NVFP4_OK) {
      fail = true;
      if (c.call() != NVFP4_EHIP) printf("%s: a rejected launch is not NVFP4_EHIP\n", c.name), ++bad;
    }
    ++n;
  }
  // workspace queries take anything
  for (int64_t x : {(int64_t)-1, (int64_t)0, (int64_t)1, big})
    for (int32_t h : {-1, 0, 8, 64, big32}) {
      nvfp4_attn_tree_workspace_bytes(x, h, h, 8, 128, x, x);
      nvfp4_attn_tree_workspace_bytes(65535, 64, h, 8, 128, 1 << 20, 0);
      nvfp4_verify_drafts_workspace_bytes(x, h, x, h);
      ++n;
    }
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

// Host-only check of the token mixers' argument handling (api_mixers.cpp), built with
// the address and undefined-behaviour sanitizers against stand-in launchers: rejected
// calls request no launch, accepted ones one, and a launch the runtime rejects comes
// back as NVFP4_EHIP.  Buffers are fake device addresses, never dereferenced; sizes go to
// the ends of their ranges, so that an overflow in a check would show.
// Prints one line per failed case and "ok <n>" at the end.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <functional>
#include <limits>
#include <string>
#include <vector>

#include "../../nvfp4_w4a4_block_act_amd/csrc/mixers.hpp"

static int launches = 0;
static bool fail = false;
static hipError_t record() {
  ++launches;
  return fail ? hipErrorLaunchFailure : hipSuccess;
}
namespace nvfp4 {
hipError_t launch_kv_append(const AppendArgs&, hipStream_t) { return record(); }
size_t attn_decode_workspace(int64_t B, int q_heads, int, int head_dim, int64_t max_len, int64_t) {
  return max_len >= 1024 ? (size_t)B * q_heads * head_dim * 4 : 0;
}
hipError_t launch_attn_decode(const AttnArgs&, hipStream_t) { return record(); }
hipError_t launch_gdn_step(const GdnArgs&, hipStream_t) { return record(); }
size_t gdn_prefill_workspace(int64_t T, int64_t B, int, int v_heads, int, int) {
  return T == 0 ? 0 : (size_t)(T / 64 + B) * v_heads * 1024;
}
hipError_t launch_gdn_prefill(const GdnArgs&, hipStream_t) { return record(); }
}  // namespace nvfp4

namespace {
template <class T = void>
T* at(uintptr_t mb, uintptr_t off = 0) {
  return reinterpret_cast<T*>((uintptr_t(1) << 40) + (mb << 20) + off);
}
nvfp4_kv_cache cache() {
  return {at(0), at(64), nullptr, nullptr, 32, 16 * 1024, 1024, 128, 16, 8, 128, NVFP4_BF16};
}
nvfp4_status append(const nvfp4_kv_cache& c, int64_t T = 4, int heads = 40, int64_t ldq = 5120, int64_t ldk = 1024,
                    int rot = 128, int64_t far = 4096) {
  return nvfp4_kv_append(at(128), at(160), at(192), NVFP4_BF16, T, heads, ldq, ldk, ldk, at<float>(224), rot, far, 0,
                         at<int64_t>(256), at<int64_t>(257), &c, at(288), ldq, nullptr);
}
nvfp4_status attn(const nvfp4_kv_cache& c, int64_t B = 4, int heads = 40, int64_t max_len = 512, int64_t ldt = 32,
                  int64_t window = 0, size_t wsb = 0, float scale = 1.0f) {
  return nvfp4_attn_decode(at(128), B, heads, 5120, &c, at<int32_t>(160), ldt, at<int32_t>(161), max_len, scale, window,
                           at(192), 5120, at<float>(224), at(256), wsb, nullptr);
}
nvfp4_status step(int64_t B = 4, int hk = 16, int hv = 32, int dk = 128, int dv = 128, int64_t states = 8,
                  const float* beta = at<float>(65)) {
  return nvfp4_gdn_step(at(0), 2048, at(16), 2048, at(32), 4096, at<float>(64), 32, beta, 32, B, hk, hv, dk, dv,
                        at<float>(128), states, at<int32_t>(67), 0.1f, at(96), 4096, nullptr);
}
nvfp4_status prompt(int64_t T = 64, int64_t B = 4, int hv = 32, int64_t states = 8, size_t wsb = 1 << 30) {
  return nvfp4_gdn_prefill(at(0), 2048, at(16), 2048, at(32), 4096, at<float>(64), 32, at<float>(65), 32, T, B,
                           at<int32_t>(66), 16, hv, 128, 128, at<float>(128), states, at<int32_t>(67), at<int32_t>(68),
                           0.1f, at(96), 4096, at(512), wsb, nullptr);
}
struct Case {
  const char* name;
  std::function<nvfp4_status()> call;
  nvfp4_status want;
};
}  // namespace

int main() {
  const int64_t big = std::numeric_limits<int64_t>::max();
  auto with = [](auto set) {
    nvfp4_kv_cache c = cache();
    set(c);
    return c;
  };
  std::vector<Case> cases = {
      {"append", [] { return append(cache()); }, NVFP4_OK},
      {"append T max", [=] { return append(cache(), big); }, NVFP4_ESHAPE},
      {"append T 2^22 + 1", [] { return append(cache(), (1 << 22) + 1); }, NVFP4_ESHAPE},
      {"append ld max", [=] { return append(cache(), 4, 40, big, 1024); }, NVFP4_ESHAPE},
      {"append ldk max", [=] { return append(cache(), 4, 40, 5120, big - 7); }, NVFP4_ESHAPE},
      {"append far max", [=] { return append(cache(), 4, 40, 5120, 1024, 128, big); }, NVFP4_ESHAPE},
      {"append heads", [] { return append(cache(), 4, 1 << 30); }, NVFP4_ESHAPE},
      {"append page stride max", [=] { return append(with([=](auto& c) { c.page_stride = big - 7; })); }, NVFP4_ESHAPE},
      {"append stride product", [=] { return append(with([](auto& c) { c.num_pages = (1LL << 31) - 1, c.page_stride = (1LL << 40) - 8; })); }, NVFP4_ESHAPE},
      {"append widest pool", [=] { return append(with([](auto& c) { c.num_pages = 1 << 16, c.page_stride = (1LL << 40) - 8, c.v = at(0, 2 * 16 * 1024); })); }, NVFP4_EINVAL},
      {"append head stride max", [=] { return append(with([](auto& c) { c.head_stride = (1LL << 40) - 8; })); }, NVFP4_EINVAL},
      {"append kv heads", [=] { return append(with([](auto& c) { c.kv_heads = std::numeric_limits<int32_t>::max(); })); }, NVFP4_ESHAPE},
      {"append page size", [=] { return append(with([](auto& c) { c.page_size = 0x7FFFFFF0; })); }, NVFP4_ESHAPE},
      {"append overlapping rows", [=] { return append(with([](auto& c) { c.token_stride = 0; })); }, NVFP4_ESHAPE},
      {"append interleaved k and v", [=] { return append(with([](auto& c) { c.page_stride = 2 * 16 * 1024, c.v = at(0, 2 * 16 * 1024); })); }, NVFP4_OK},
      {"append empty pool", [=] { return append(with([](auto& c) { c.num_pages = 0, c.k = c.v = nullptr; })); }, NVFP4_OK},
      {"attn", [] { return attn(cache()); }, NVFP4_OK},
      {"attn empty pool", [=] { return attn(with([](auto& c) { c.num_pages = 0, c.k = c.v = nullptr; })); }, NVFP4_OK},
      {"attn max_len max", [=] { return attn(cache(), 4, 40, big, big); }, NVFP4_ESHAPE},
      {"attn window max", [=] { return attn(cache(), 4, 40, 512, 32, big); }, NVFP4_ESHAPE},
      {"attn B max", [=] { return attn(cache(), big); }, NVFP4_ESHAPE},
      {"attn launch too large", [] { return attn(cache(), 65535, 80); }, NVFP4_ESHAPE},
      {"attn heads max", [] { return attn(cache(), 4, 0x7FFFFFF8); }, NVFP4_ESHAPE},
      {"attn workspace", [] { return attn(cache(), 4, 40, 2048, 128, 0, 16); }, NVFP4_EWORKSPACE},
      {"attn nan scale", [] { return attn(cache(), 4, 40, 512, 32, 0, 0, std::nanf("")); }, NVFP4_EINVAL},
      {"step", [] { return step(); }, NVFP4_OK},
      {"step without beta", [] { return step(4, 16, 32, 128, 128, 8, nullptr); }, NVFP4_OK},
      {"step B max", [=] { return step(big); }, NVFP4_ESHAPE},
      {"step launch too large", [] { return step(65535, 16, 32, 128, 128, 1 << 20); }, NVFP4_ESHAPE},
      {"step states max", [=] { return step(4, 16, 32, 128, 128, big); }, NVFP4_ESHAPE},
      {"step heads max", [] { return step(4, 0x7FFFFFFF, 0x7FFFFFFF); }, NVFP4_ESHAPE},
      {"step state over out", [] { return step(4, 16, 32, 128, 128, (1LL << 31) - 1); }, NVFP4_OK},
      {"prompt", [] { return prompt(); }, NVFP4_OK},
      {"prompt T max", [=] { return prompt(big); }, NVFP4_ESHAPE},
      {"prompt T 2^28 + 64", [] { return prompt((1 << 28) + 64); }, NVFP4_ESHAPE},
      {"prompt T 2^27, two value heads to a key head", [] { return prompt(1 << 27); }, NVFP4_ESHAPE},
      {"prompt workspace", [] { return prompt(4096, 4, 32, 8, 1024); }, NVFP4_EWORKSPACE},
      {"prompt no sequences", [] { return prompt(64, 0); }, NVFP4_OK},
  };
  int bad = 0, n = 0;
  for (const Case& c : cases) {
    launches = 0;
    fail = false;
    const nvfp4_status s = c.call();
    const bool none = std::string(c.name) == "prompt no sequences";
    if (s != c.want || launches != (s == NVFP4_OK && !none ? 1 : 0)) {
      printf("%s: status %d (want %d), %d launches\n", c.name, s, c.want, launches);
      ++bad;
    }
    if (c.want == NVFP4_OK && !none) {
      fail = true;
      if (c.call() != NVFP4_EHIP) printf("%s: a rejected launch is not NVFP4_EHIP\n", c.name), ++bad;
    }
    ++n;
  }
  // workspace queries take anything
  for (int64_t x : {(int64_t)-1, (int64_t)0, (int64_t)1, big})
    for (int32_t h : {-1, 0, 8, 0x7FFFFFFF}) {
      nvfp4_attn_decode_workspace_bytes(x, h, 8, 128, x, x);
      nvfp4_gdn_prefill_workspace_bytes(x, x, h, h, 128, 128);
      ++n;
    }
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

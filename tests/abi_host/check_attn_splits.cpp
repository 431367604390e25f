// Host-only check of the decode attention's split rule (attn_splits.hpp): a launch's splits
// cover every sequence up to the bound, sequences near the bound get the host's own split,
// and a loose bound leaves a sequence about as many splits as a tight one.  Prints one line
// per failed case and "ok <n>" at the end.
#include <cmath>
#include <cstdio>
#include <random>

#include "../../nvfp4_w4a4_block_act_amd/csrc/attn_splits.hpp"

using namespace nvfp4;

int main() {
  int bad = 0, n = 0;
  std::mt19937 rng(1);
  auto log_uniform = [&](double low, double high) {
    return (int)(low * pow(high / low, std::uniform_real_distribution<double>(0, 1)(rng)));
  };
  auto fail = [&](const char* what, int rows, int len, int max_len, int window, Splits s, int tokens) {
    if (bad++ < 20)
      printf("%s: rows %d length %d bound %d window %d: %d splits of %d, own %d\n", what, rows, len, max_len, window, s.count,
             s.tokens, tokens);
  };
  for (int i = 0; i < 400000; ++i) {
    const int rows = log_uniform(1, 3200), len = i % 50 ? log_uniform(1, 1 << 30) : 0;
    const int max_len = i % 4 == 0 && len > 0 ? len : log_uniform(len + 1, 1 << 30);
    const int window = i % 3 ? 0 : log_uniform(1, (1u << 31) - 1);
    const Splits room = attn_splits(rows, max_len, window);
    if (room.count < 1 || room.tokens < 16 || room.tokens % 16 ||
        (int64_t)room.count * room.tokens < attn_span(max_len, window))
      fail("host", rows, len, max_len, window, room, 0);
    if (room.count == 1) continue;  // (one split takes all there is)
    const int64_t span = attn_span(len, window), bound = attn_span(max_len, window);
    const int tokens = attn_split_tokens(rows, room.tokens, (int)bound, (int)span);
    if (tokens < 16 || tokens % 16 || tokens > room.tokens || (int64_t)tokens * room.count < span)
      fail("cover", rows, len, max_len, window, room, tokens);
    // a split's first token and end stay inside 32 bits
    if ((int64_t)len - span + (int64_t)(room.count + 1) * tokens > 0x7FFFFFFF)
      fail("past 2^31", rows, len, max_len, window, room, tokens);
    if (2 * span > bound && tokens > 512 && tokens != room.tokens) fail("near", rows, len, max_len, window, room, tokens);
    // as many workgroups as under a tight bound, but for the part of a half that the bound is
    // away from a power of two times the length
    const Splits tight = attn_splits(rows, len > 0 ? len : 1, window);
    const int64_t live = (span + tokens - 1) / tokens;
    if (2 * live + 1 < tight.count) fail("few", rows, len, max_len, window, room, tokens);
    ++n;
  }
  // 16 sequences of 4096 on 8 key-value heads, one of 4096: as many splits as with the tight bound
  for (const int rows : {128, 8})
    for (int max_len = 4096; max_len <= 1 << 20; max_len *= 2) {
      const Splits room = attn_splits(rows, max_len, 0), tight = attn_splits(rows, 4096, 0);
      const int tokens = attn_split_tokens(rows, room.tokens, max_len, 4096);
      if (tokens != tight.tokens) fail("pinned", rows, 4096, max_len, 0, room, tokens);
    }
  if (bad) return 1;
  printf("ok %d\n", n);
  return 0;
}

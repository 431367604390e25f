// How the decode attention splits a sequence's tokens over workgroups.  The host takes the
// number of splits of a launch from the bound of the lengths; the kernels take a sequence's
// share of them from its own length, so that a loose bound only adds workgroups without work.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <algorithm>

#include "launch.hpp"

namespace nvfp4 {

// Splits of a sequence, from sizes the host knows: about twelve workgroups for each CU
// (uneven lengths even out over them), none with fewer than 512 tokens -- or 256 where
// there would be less than two workgroups for each CU, but no split, and no second
// kernel, for less than 1024.  8 heads of 128, E4M3, against eight and sixteen for each CU: 67
// sequences of up to 4099 take 9 % and 3 % less time, 128 of up to 4096 2 % less and 3 % more,
// 160 of up to 1024 2 % more and as much.  24 of up to 2000, 4 heads of 256 in bf16, take 30 %
// more with splits of 512, one of 32768 15 % more with splits of 256.  Equal shares of all
// sequences' tiles, as many as the GPU holds at once, taken from the lengths on the device,
// were no faster, and a fifth slower for one of 32768.
struct Splits {
  int count, tokens;  // tokens of one split: a multiple of 16
};

// Tokens that a sequence's splits cover at most: from the tile that the window begins in.
__host__ __device__ inline int64_t attn_span(int64_t len, int64_t window) {
  return window > 0 && window < len ? window + 15 : len;
}

// rows: workgroups of one split, (sequence, key-value head, 16 of its query heads).
inline Splits attn_splits(int64_t rows, int64_t max_len, int64_t window) {
  const int64_t span = attn_span(max_len, window);
  const int64_t want = std::max<int64_t>(1, (int64_t)kCUs * 12 / rows);
  int64_t n = std::min(want, std::max<int64_t>(1, span / 512));
  if (n > 1 && rows * n < 2 * kCUs) n = std::min((2 * kCUs + rows - 1) / rows, span / 256);
  const int64_t tokens = std::max<int64_t>(16, (span + n - 1) / n + 15) / 16 * 16;
  return {(int)std::max<int64_t>(1, (span + tokens - 1) / tokens), (int)tokens};
}

// Tokens of a split of one sequence, in a launch whose splits (more than one) of `tokens`
// each cover `bound` tokens: where the sequence's span is at most a half, a quarter, ... of
// the bound, the like part of them, but not less than 512 -- or 256 where the rows would have
// less than two workgroups for each CU if all were as long.  16 sequences of 4096 (E4M3, 8 heads
// of 128) take 32 us under a bound of 4096 and 33 under 131072 (61 with the bound's own splits),
// one of 4096 13 under 4096 and under 2^20 (35), 67 of 1024 to 4099 76 and 76 (104); uneven
// lengths under a tight bound lose or gain up to 3 % (128 of 1024 to 4096 133 us against 130,
// 40 of 2048 to 8192 85 against 87).  The splits of a tight bound, found from the longest length
// on the device, cost every workgroup its search: 3 to 10 % under tight bounds.
__host__ __device__ inline int attn_split_tokens(int rows, int tokens, int bound, int span) {
  int halves = 0;
  if (span > 0 && span <= bound) halves = __builtin_clz(span) - __builtin_clz(bound);
  if (halves > 0 && (int64_t)span << halves > bound) --halves;
  const int share = (((tokens - 1) >> halves) + 16) / 16 * 16;
  const int64_t spread = (int64_t)rows * span / (2 * kCUs);  // a workgroup's tokens with two for each CU
  const int least = spread >= 512 ? 512 : (spread <= 256 ? 256 : ((int)spread + 15) / 16 * 16);
  return share >= tokens || least >= tokens ? tokens : (share > least ? share : least);
}

}  // namespace nvfp4

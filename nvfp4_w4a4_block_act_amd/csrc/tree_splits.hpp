// How the tree attention splits a sequence's tokens over workgroups, by the rules of the
// decode attention (attn_splits.hpp): the host takes the number of splits of a launch from
// the bound of the lengths, the kernels a sequence's share of them from its own length.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <algorithm>

#include "attn_splits.hpp"

namespace nvfp4 {

constexpr int kTreeTile = 32;  // tokens

// Tokens from the tile in which a sequence's attended context begins to its last drafted one.
__host__ __device__ inline int64_t tree_span(int64_t ctx, int64_t nodes, int64_t window) {
  return (window > 0 && window < ctx ? window + kTreeTile - 1 : ctx) + nodes;
}

// rows: workgroups of one split.  About six workgroups for each CU, of which one or two run at once: 6 sequences of
// up to 32768, 64 nodes, 6 heads of 256 on each of 4 (one at once), take 444 us, 470 with three, 454 with four, 481
// with eight and 530 with twelve; 48 of up to 4099, 16 nodes, 5 heads on each of 8 (two), 143, 153, 153, 145 and 150.
inline Splits tree_splits(int64_t rows, int64_t max_len, int64_t nodes, int64_t window) {
  const int64_t span = tree_span(max_len, nodes, window);
  const int64_t want = std::max<int64_t>(1, (int64_t)kCUs * 6 / rows);
  int64_t n = std::min(want, std::max<int64_t>(1, span / 512));
  if (n > 1 && rows * n < 2 * kCUs) n = std::min((2 * kCUs + rows - 1) / rows, span / 256);
  const int64_t tokens = (std::max<int64_t>(1, (span + n - 1) / n) + kTreeTile - 1) / kTreeTile * kTreeTile;
  return {(int)((span + tokens - 1) / tokens), (int)tokens};
}

// Tokens of a split of one sequence of `span`, where the launch's bound of it is `bound`.
__host__ __device__ inline int tree_split_tokens(int rows, int tokens, int bound, int span) {
  const int t = (attn_split_tokens(rows, tokens, bound, span) + kTreeTile - 1) / kTreeTile * kTreeTile;
  return t < tokens ? t : tokens;
}

}  // namespace nvfp4

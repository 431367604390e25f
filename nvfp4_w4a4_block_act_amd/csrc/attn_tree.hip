// Attention for a tree of drafted tokens over the paged key-value cache.
//
// The rows of a key-value head are the nodes of the tree times the query heads that share
// it: up to 64 x (query heads / key-value heads).  As in the decode attention there is one pass over the
// tokens, with a running reference m and sum l of each row's softmax, scores in units of
// log 2, and m moves only when a score exceeds it by more than kSlack.
//
// Layout.  A wave takes NR blocks of 16 rows and tiles of 32 tokens; RW waves share a
// tile, each with rows of its own, and KW such groups of waves take tiles in turn, with the
// same rows, joined through LDS at the end.  Keys and values pass through LDS as bf16 rows
// (E4M3 codes widen exactly on the way in): whole rows are loaded side by side, the next
// tile's while one is computed.
//  * scores: S^T = K Q^T (16 x 16 x 32): lane (r, g) = (lane % 16, lane / 16) takes 16-byte
//    pieces of token r's key row, and one read of a piece serves the wave's NR blocks;
//  * S^T leaves token 16 s + 4 g + j of row r in register (s, j) of lane (r, g): as element
//    4 s + j of a lane's eight these are an operand of O^T = V^T P^T (16 x 16 x 32) in place;
//  * V^T: lane (c, g) takes its head_dim / 16 elements of the value rows of those eight tokens,
//    and the transposition is byte permutes within the lane, once for the NR blocks.
// A weight enters as the sum of two bf16 values (16 significant bits).
//
// Masks: the ancestors of a node are a word of 64 bits that the wave forms from the parents by
// doubling; only tiles that hold drafted tokens, or the edge of a window, or a page outside
// the pool, look at it.  In these tiles values that are no finite number are taken as 0, so
// that a node's row that holds one does not reach the rows that do not see it.
#include <algorithm>

#include "common.hpp"
#include "drafts.hpp"
#include "mixers_device.hpp"
#include "tree_splits.hpp"

namespace nvfp4 {
namespace {

constexpr float kNone = -3.402823466e38f;  // reference before any token: finite, so that differences are numbers
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// How a launch splits its sequences, as the kernels get it.
struct Plan {
  int rows, blocks, splits, tokens, bound;  // blocks: workgroups that share a key-value head's rows
  __device__ __forceinline__ int tokens_of(int span) const {
    return splits == 1 ? tokens : tree_split_tokens(rows, tokens, bound, span);
  }
};

// Where a sequence's tiles begin, and the tokens from there on.
struct Range {
  int ctx, begin, span;
};
__device__ __forceinline__ Range range_of(const TreeArgs& a, int b) {
  const int ctx = min(max(a.lens[b], 0), a.max_len);
  const int begin = a.window > 0 && a.window < ctx ? (ctx - a.window) / kTreeTile * kTreeTile : 0;
  return {ctx, begin, ctx + a.nodes - begin};
}

template <int DIM, bool FP8>
struct Shape {
  static constexpr int kRow = DIM * (FP8 ? 1 : 2);  // bytes of a cache row
  static constexpr int kLanes = kRow / 16;
  static constexpr int kLdsRow = DIM * 2 + 16;      // 16 rows' pieces fall on different banks
  static constexpr int kLdsTile = 2 * kTreeTile * kLdsRow;
};

__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

__device__ __forceinline__ bf16x8_t octet(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(a, b, c, d));
}

// Two bf16 values, 0 for one that is no finite number.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// Nodes on each lane's way to the context, itself included; 0 for a padded node.
__device__ __forceinline__ uint64_t ancestors(const TreeArgs& a, int b, int lane) {
  if (!a.parents) return lane < a.nodes ? ~0ull >> (63 - lane) : 0;
  int up = lane < a.nodes ? a.parents[(int64_t)b * a.nodes + lane] : -2;
  if (up < -1 || up >= lane) up = -2;
  uint64_t seen = 1ull << lane;
  for (int s = 1; s < a.nodes; s *= 2) {
    const int at = max(up, 0);
    const uint32_t lo = __shfl((uint32_t)seen, at), hi = __shfl((uint32_t)(seen >> 32), at);
    const int next = __shfl(up, at);
    if (up >= 0) seen |= (uint64_t)hi << 32 | lo, up = next;
  }
  return up == -1 ? seen : 0;
}

__device__ __forceinline__ int64_t part_row(const TreeArgs& a, int64_t row, int splits, int s) { return row * splits + s; }

template <int DIM, bool FP8, int NR, int RW, int KW>
__global__ __launch_bounds__(RW* KW * 64, 2) void attn_tree_kernel(TreeArgs a, Plan plan) {
  using Sh = Shape<DIM, FP8>;
  constexpr int ES = FP8 ? 1 : 2, PAD = DIM + 4, kRows = NR * RW * 16, kWaves = RW * KW;
  constexpr int kLoads = Sh::kLanes / RW;        // pieces of a lane: 64 rows (keys, values) over RW waves
  constexpr int kStep = 64 * RW / Sh::kLanes;    // rows that a piece of each lane spans
  static_assert(kLoads >= 1, "a wave's share of a tile");
  const nvfp4_kv_cache& c = a.cache;
  const int splits = plan.splits, group = a.q_heads / c.kv_heads;
  const int gx = c.kv_heads * plan.blocks;
  // the workgroups of one split run side by side on one XCD: the tiles come from its cache
  const uint32_t turn = blockIdx.x / 8, which = turn % gx, item = (turn / gx) * 8 + blockIdx.x % 8;
  const int kvh = which / plan.blocks, block = which % plan.blocks;
  const int b = item / splits, split = (item % splits + b / (8 / min(8, splits & -splits))) % splits;
  if (b >= a.B) return;
  const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), rw = wave % RW, kw = wave / RW;

  const Range range = range_of(a, b);
  const int split_tokens = plan.tokens_of(range.span);
  const int from = range.begin + split * split_tokens, end = range.ctx + a.nodes;
  const int to = min(end, from + split_tokens);
  const bool only = split_tokens >= range.span;  // the sequence has one split: no join
  if (split > 0 && from >= end) return;

  // rows: node * group + head, blocks of 16 to a wave
  const int all_rows = a.nodes * group, row0 = block * kRows + rw * NR * 16;
  const uint64_t anc_lane = ancestors(a, b, lane);
  uint64_t anc[NR];
  int low[NR];  // first token of the context that the row sees
  bf16x8_t q[NR][DIM / 32];
  bool any = false;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int row = row0 + n * 16 + r, node = min(row, all_rows - 1) / group, head = min(row, all_rows - 1) % group;
    const uint32_t lo = __shfl((uint32_t)anc_lane, node), hi = __shfl((uint32_t)(anc_lane >> 32), node);
    anc[n] = (uint64_t)hi << 32 | lo;
    low[n] = 0;
    any |= anc[n] != 0 && row < all_rows;
    if (a.window > 0 && anc[n]) {
      int own = __popcll(anc[n]);
      for (; own > a.window; --own) anc[n] &= anc[n] - 1;  // the farthest ancestors
      low[n] = max(0, range.ctx - (a.window - own));
    }
    const uint16_t* qp = a.q + ((int64_t)b * a.nodes + node) * a.ldq + (int64_t)(kvh * group + head) * DIM;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i) q[n][i] = *reinterpret_cast<const bf16x8_t*>(qp + i * 32 + g * 8);
  }
  const float factor = a.scale * (FP8 ? *c.k_amax / 448.0f : 1.0f) * kLog2e;
  // tiles below hold tokens that some row's window leaves out
  const int edge = a.window > 0 ? max(0, range.ctx - max(0, a.window - a.nodes)) : 0;

  extern __shared__ float4_t dynamic_lds[];
  uint8_t* corner = reinterpret_cast<uint8_t*>(dynamic_lds) + kw * Sh::kLdsTile;
  float m[NR], l[NR];
  float4_t o[NR][DIM / 16];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    m[n] = kNone, l[n] = 0;
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) o[n][i] = {0, 0, 0, 0};
  }

  // tiles from / 32 + kw + KW * n, as many turns for all waves (barriers where waves share a tile)
  const int tile0 = from / kTreeTile, tile_end = (to + kTreeTile - 1) / kTreeTile;
  const bool work = RW > 1 ? __syncthreads_or(any) : __any(any);
  const int turns = work && tile0 < tile_end && c.num_pages > 0 ? (tile_end - tile0 + KW - 1) / KW : 0;
  const uint8_t* kc = static_cast<const uint8_t*>(c.k) + (int64_t)kvh * c.head_stride * ES;
  const uint8_t* vc = static_cast<const uint8_t*>(c.v) + (int64_t)kvh * c.head_stride * ES;
  const int member = rw * 64 + lane;  // of the RW waves that load a tile
  const uint32_t stride = (uint32_t)c.token_stride * ES;
  const int half_last = (end - 1) / 16;  // the last 16 tokens' half tile

  u32x4_t held[kLoads];
  bool outside[2];  // the half's page is not in the pool
  auto fetch = [&](int tile) {
    int64_t at[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int half = min(tile * 2 + s, half_last), token = half * 16, page_index = token / c.page_size;
      const int page = a.table[(int64_t)b * a.ldt + page_index];
      outside[s] = page < 0 || page >= c.num_pages;
      at[s] = ((int64_t)(outside[s] ? 0 : page) * c.page_stride + (int64_t)(token - page_index * c.page_size) * c.token_stride) * ES;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kStep + member / Sh::kLanes;  // keys 0 .. 31, values 32 .. 63
      const uint8_t* base = (row < 32 ? kc : vc) + ((row & 16) ? at[1] : at[0]);
      held[i] = *reinterpret_cast<const u32x4_t*>(base + ((uint32_t)(row & 15) * stride + member % Sh::kLanes * 16));
    }
  };
  auto put = [&](bool masked) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kStep + member / Sh::kLanes;
      uint32_t w[FP8 ? 8 : 4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (FP8)
          w[2 * x] = fp8_pair(held[i][x], false), w[2 * x + 1] = fp8_pair(held[i][x], true);
        else
          w[x] = held[i][x];
      }
      if (masked && row >= 32) {
#pragma unroll
        for (int x = 0; x < (FP8 ? 8 : 4); ++x) w[x] = finite_pair(w[x]);
      }
      uint8_t* to_lds = corner + row * Sh::kLdsRow + member % Sh::kLanes * (FP8 ? 32 : 16);
      *reinterpret_cast<uint4*>(to_lds) = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (FP8) *reinterpret_cast<uint4*>(to_lds + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  };
  auto share = [&] {
    if constexpr (RW > 1)
      __syncthreads();
    else
      wave_lds_fence();
  };

  if (turns > 0) fetch(min(tile0 + kw, tile_end - 1));
  for (int turn_of = 0; turn_of < turns; ++turn_of) {
    const int tile = tile0 + kw + turn_of * KW, start = tile * kTreeTile;
    const bool mine = tile < tile_end;  // the last turn may have fewer tiles than groups
    const bool gone[2] = {outside[0], outside[1]};
    const bool masked = start + kTreeTile > range.ctx || start < edge || gone[0] || gone[1];
    put(masked);
    share();
    if (turn_of + 1 < turns) fetch(min(tile + KW, tile_end - 1));
    if (mine) {
      float4_t s[NR][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][h] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < DIM / 32; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(corner + (h * 16 + r) * Sh::kLdsRow + i * 64 + g * 16);
          const bf16x8_t k = octet(w.x, w.y, w.z, w.w);
#pragma unroll
          for (int n = 0; n < NR; ++n) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][i], s[n][h], 0, 0, 0);
        }
      }
      bf16x8_t hi[NR], lo[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s[n][e / 4][e % 4] * factor;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int t = start + e / 4 * 16 + g * 4 + e % 4, drafted = t - range.ctx;
            const bool seen = drafted < 0 ? t >= low[n] : drafted < 64 && (anc[n] >> drafted & 1);
            if (!seen || gone[e / 4]) x[e] = -INFINITY;
          }
        }
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if (__any(top > m[n] + kSlack)) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m[n]);
          const float keep = __builtin_amdgcn_exp2f(m[n] - top);
          m[n] = top;
          l[n] *= keep;
#pragma unroll
          for (int i = 0; i < DIM / 16; ++i) o[n][i] *= keep;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(x[e] - m[n]);
          l[n] += x[e];
        }
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hw[e] = bf16_pair(x[2 * e], x[2 * e + 1]);
          lw[e] = bf16_pair(x[2 * e] - __uint_as_float(hw[e] << 16), x[2 * e + 1] - __uint_as_float(hw[e] & 0xFFFF0000u));
        }
        hi[n] = octet(hw[0], hw[1], hw[2], hw[3]);
        lo[n] = octet(lw[0], lw[1], lw[2], lw[3]);
      }
      // values: tokens 16 s + 4 g + j in runs of 16 bytes at most
      constexpr int kRun = DIM < 128 ? DIM / 32 : 4, kRuns = DIM / 32 / kRun;  // dwords of a run; runs of a row
#pragma unroll
      for (int u = 0; u < kRuns; ++u) {
        uint32_t v[8][kRun];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint8_t* p = corner + (32 + e / 4 * 16 + g * 4 + e % 4) * Sh::kLdsRow + u * 256 + r * kRun * 4;
          if constexpr (kRun == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            v[e][0] = w.x, v[e][1] = w.y;
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            v[e][0] = w.x, v[e][1] = w.y, v[e][2] = w.z, v[e][3] = w.w;
          }
        }
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
          const bf16x8_t even = octet(low_halves(v[0][x], v[1][x]), low_halves(v[2][x], v[3][x]),
                                      low_halves(v[4][x], v[5][x]), low_halves(v[6][x], v[7][x]));
          const bf16x8_t odd = octet(high_halves(v[0][x], v[1][x]), high_halves(v[2][x], v[3][x]),
                                     high_halves(v[4][x], v[5][x]), high_halves(v[6][x], v[7][x]));
          const int i = (u * kRun + x) * 2;
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, lo[n], o[n][i], 0, 0, 0);
            o[n][i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, lo[n], o[n][i + 1], 0, 0, 0);
            o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, hi[n], o[n][i], 0, 0, 0);
            o[n][i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, hi[n], o[n][i + 1], 0, 0, 0);
          }
        }
      }
    }
    share();
  }

  // the groups' results, joined in LDS
  __shared__ float ms[kWaves][NR * 16], ls[kWaves][NR * 16];
  float* os = reinterpret_cast<float*>(dynamic_lds);  // [group][kRows][PAD], over the tiles
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    if (anc[n] == 0) {  // a padded node: the tiles of the context have no mask
      m[n] = kNone, l[n] = 0;
#pragma unroll
      for (int i = 0; i < DIM / 16; ++i) o[n][i] = {0, 0, 0, 0};
    }
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
    if (g == 0) ms[wave][n * 16 + r] = m[n], ls[wave][n * 16 + r] = l[n];
    // element of the row that output tile i holds in row 4 g + j: value rows are read in runs of 16 bytes at most
    constexpr int kEach = DIM == 256 ? 8 : DIM / 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < DIM / 16; i += 4) {
        const int at = i / kEach * 128 + (g * 4 + j) * kEach + i % kEach;
        const float4_t w = {o[n][i][j], o[n][i + 1][j], o[n][i + 2][j], o[n][i + 3][j]};
        *reinterpret_cast<float4_t*>(os + (kw * kRows + (rw * NR + n) * 16 + r) * PAD + at) = w;
      }
  }
  __syncthreads();
  const float vg = FP8 ? *c.v_amax / 448.0f : 1.0f;
  float* parts = static_cast<float*>(a.workspace);
  const int64_t rows = (int64_t)a.B * a.nodes * a.q_heads;
  float2* ml = reinterpret_cast<float2*>(parts + rows * splits * DIM);
  const int mine_rows = min(kRows, all_rows - block * kRows);
  for (int e = threadIdx.x * 4; e < mine_rows * DIM; e += kWaves * 64 * 4) {
    const int row = e / DIM, d = e % DIM, w0 = row / (NR * 16), in = row % (NR * 16);
    float top = kNone, sum = 0;
#pragma unroll
    for (int w = 0; w < KW; ++w) top = fmaxf(top, ms[w * RW + w0][in]);
    float4_t x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float f = __builtin_amdgcn_exp2f(ms[w * RW + w0][in] - top);
      sum += ls[w * RW + w0][in] * f;
      x += *reinterpret_cast<const float4_t*>(os + (w * kRows + row) * PAD + d) * f;
    }
    const int node = (block * kRows + row) / group, head = kvh * group + (block * kRows + row) % group;
    const int64_t token = (int64_t)b * a.nodes + node;
    if (only) {
      const float4_t y = x * (sum == 0 ? 0.0f : vg / sum);
      *reinterpret_cast<uint2*>(a.out + token * a.ldo + (int64_t)head * DIM + d) = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
      if (a.lse && d == 0) a.lse[token * a.q_heads + head] = sum == 0 ? -INFINITY : top * kLn2 + logf(sum);
    } else {
      const int64_t at = part_row(a, token * a.q_heads + head, splits, split);
      *reinterpret_cast<float4_t*>(parts + at * DIM + d) = x;
      if (d == 0) ml[at] = make_float2(top, sum);
    }
  }
}

// Joins the splits of one row: each counts 2^(its m - the largest m).  Groups of DIM / 4
// threads take the splits in turn, then one group their sums.
template <int DIM, bool FP8, int kGroups>
__global__ __launch_bounds__(DIM / 4 * kGroups) void tree_join_kernel(TreeArgs a, Plan plan) {
  constexpr int kLanes = DIM / 4;
  const int splits = plan.splits;
  const int64_t row = blockIdx.x, token = row / a.q_heads;
  const int head = (int)(row % a.q_heads), d = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const Range range = range_of(a, (int)(token / a.nodes));
  const int split_tokens = plan.tokens_of(range.span), used = (range.span + split_tokens - 1) / split_tokens;
  if (used <= 1) return;
  const float* parts = static_cast<const float*>(a.workspace);
  const float2* ml = reinterpret_cast<const float2*>(parts + (int64_t)a.B * a.nodes * a.q_heads * splits * DIM) +
                     part_row(a, row, splits, 0);
  const float* x_row = parts + part_row(a, row, splits, 0) * DIM + d * 4;
  float m = kNone, sum = 0;
  float4_t x = {0, 0, 0, 0};
  for (int s = grp; s < used; s += kGroups) {
    const float2 w = ml[s];
    const float4_t v = *reinterpret_cast<const float4_t*>(x_row + (int64_t)s * DIM);
    const float top = fmaxf(m, w.x), keep = __builtin_amdgcn_exp2f(m - top), f = __builtin_amdgcn_exp2f(w.x - top);
    m = top;
    sum = sum * keep + w.y * f;
    x = x * keep + v * f;
  }
  __shared__ float ms[kGroups], ls[kGroups];
  __shared__ float4_t xs[kGroups][kLanes];
  xs[grp][d] = x;
  if (d == 0) ms[grp] = m, ls[grp] = sum;
  __syncthreads();
  if (grp > 0) return;
  float top = kNone;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) top = fmaxf(top, ms[i]);
  sum = 0, x = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float f = __builtin_amdgcn_exp2f(ms[i] - top);
    sum += ls[i] * f;
    x += xs[i][d] * f;
  }
  x = x * (sum == 0 ? 0.0f : (FP8 ? *a.cache.v_amax / 448.0f : 1.0f) / sum);
  *reinterpret_cast<uint2*>(a.out + token * a.ldo + (int64_t)head * DIM + d * 4) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
  if (a.lse && d == 0) a.lse[row] = sum == 0 ? -INFINITY : top * kLn2 + logf(sum);
}

// Rows of a workgroup, by the rows of a key-value head.
int wg_rows(int64_t rows, int dim) {
  if (dim == 256) return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
}

Plan tree_plan(int64_t B, int nodes, int q_heads, int kv_heads, int dim, int64_t max_len, int64_t window) {
  const int64_t rows = (int64_t)nodes * (q_heads / kv_heads), per = wg_rows(rows, dim);
  const int64_t blocks = (rows + per - 1) / per, each = B * kv_heads * blocks;
  const Splits s = tree_splits(each, max_len, nodes, window);
  return {(int)each, (int)blocks, s.count, s.tokens, (int)tree_span(max_len, nodes, window)};
}

template <int DIM, bool FP8, int NR, int RW, int KW>
hipError_t launch_rows(const TreeArgs& a, const Plan& plan, hipStream_t stream) {
  constexpr size_t lds = std::max<size_t>((size_t)KW * Shape<DIM, FP8>::kLdsTile, (size_t)KW * NR * RW * 16 * (DIM + 4) * sizeof(float));
  hipError_t e = hipSuccess;
  if (lds > 48 * 1024)  // the same for every call, from whatever thread
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_tree_kernel<DIM, FP8, NR, RW, KW>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((int64_t)a.cache.kv_heads * plan.blocks * (((int64_t)a.B * plan.splits + 7) / 8 * 8)));
  attn_tree_kernel<DIM, FP8, NR, RW, KW><<<grid, RW * KW * 64, lds, stream>>>(a, plan);
  return hipGetLastError();
}

template <int DIM, bool FP8>
hipError_t launch_dim(const TreeArgs& a, hipStream_t stream) {
  const Plan plan = tree_plan(a.B, a.nodes, a.q_heads, a.cache.kv_heads, DIM, a.max_len, a.window);
  hipError_t e;
  const int rows = wg_rows((int64_t)a.nodes * (a.q_heads / a.cache.kv_heads), DIM);
  if constexpr (DIM == 256) {
    e = rows == 16   ? launch_rows<DIM, FP8, 1, 1, 4>(a, plan, stream)
        : rows == 32 ? launch_rows<DIM, FP8, 1, 2, 2>(a, plan, stream)
                     : launch_rows<DIM, FP8, 1, 4, 1>(a, plan, stream);
  } else {
    e = rows == 16   ? launch_rows<DIM, FP8, 1, 1, 4>(a, plan, stream)
        : rows == 32 ? launch_rows<DIM, FP8, 2, 1, 4>(a, plan, stream)
        : rows == 64 ? launch_rows<DIM, FP8, 2, 2, 2>(a, plan, stream)
                     : launch_rows<DIM, FP8, 2, 4, 1>(a, plan, stream);
  }
  if (e != hipSuccess || plan.splits == 1) return e;
  const dim3 grid((unsigned)((int64_t)a.B * a.nodes * a.q_heads));
  if (plan.splits <= 16)
    tree_join_kernel<DIM, FP8, 4><<<grid, DIM, 0, stream>>>(a, plan);
  else
    tree_join_kernel<DIM, FP8, 16><<<grid, DIM * 4, 0, stream>>>(a, plan);
  return hipGetLastError();
}

}  // namespace

size_t attn_tree_workspace(int64_t B, int nodes, int q_heads, int kv_heads, int head_dim, int64_t max_len, int64_t window) {
  const int splits = tree_plan(B, nodes, q_heads, kv_heads, head_dim, max_len, window).splits;
  return splits > 1 ? (size_t)B * nodes * q_heads * splits * (head_dim + 2) * sizeof(float) : 0;
}

hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t stream) {
  const bool fp8 = a.cache.dtype == NVFP4_E4M3;
  switch (a.cache.head_dim) {
    case 64: return fp8 ? launch_dim<64, true>(a, stream) : launch_dim<64, false>(a, stream);
    case 128: return fp8 ? launch_dim<128, true>(a, stream) : launch_dim<128, false>(a, stream);
    default: return fp8 ? launch_dim<256, true>(a, stream) : launch_dim<256, false>(a, stream);
  }
}

}  // namespace nvfp4

// Attention for a tree of drafted tokens over the paged key-value cache.
//
// The rows of a key-value head are the nodes of the tree times the query heads that share
// it: up to 64 x (query heads / key-value heads).  As in the decode attention there is one pass over the
// tokens, with a running reference m and sum l of each row's softmax, scores in units of
// log 2, and m moves only when a weight 2^(s - m) is above kMost.
//
// Layout.  A wave takes NR blocks of 16 rows and tiles of 32 tokens; RW waves share a
// tile, each with rows of its own, and KW such groups of waves take tiles in turn, with the
// same rows, joined through LDS at the end.  Keys and values pass through LDS in 16 bits:
// whole rows are loaded side by side, and lie there so that no access meets a bank twice.
//  * scores: S^T = K Q^T (16 x 16 x 32): lane (r, g) = (lane % 16, lane / 16) takes 16-byte
//    pieces of token r's key row, and one read of a piece serves the wave's NR blocks;
//  * S^T leaves token 16 s + 4 g + j of row r in register (s, j) of lane (r, g): as element
//    4 s + j of a lane's eight these are an operand of O^T = V^T P^T (16 x 16 x 32) in place;
//  * V^T: lane (c, g) takes its head_dim / 16 elements of the value rows of those eight tokens,
//    and the transposition is byte permutes within the lane, once for the NR blocks;
//  * the sum of the weights is one more row of that product, of ones.
// A weight enters as the sum of two bf16 values (16 significant bits, of small ones too; two
// matrix instructions); E4M3 codes widen to bf16 exactly.  (One fp16 value over E4M3, 126 us instead of 141 for
// 48 x 16, has 11 bits, which the logarithm of their sum shows, and loses weights below 2^-25 of the largest,
// which are a part of the result in long contexts.)
// Where waves share a tile, the scores of the next one are formed while this one's weights are.
//
// Masks: the ancestors of a node are 64 bits that the wave forms from the parents by
// doubling; only tiles that hold drafted tokens, or the edge of a window, or a page outside
// the pool, look at it.  In these tiles values that are no finite number are taken as 0, so
// that a node's row that holds one does not reach the rows that do not see it; where any
// was, the rows that do see it get it at the end (the check for that takes 0.6 us of 15, 3 of 143; a call in which
// each sequence has one up to 1.8 times as long -- of padded nodes' rows, which may hold anything, it asks nothing).
//
// Bound by memory for few rows, by each wave's chain of steps in a tile for many: 48 sequences of up to 4099
// (E4M3, 5 heads on each of 8, 250 MB) take 55 us with 3 nodes (4.3 TB/s), 75 with 6, 107 with 12 and 141 with
// 16 (80 rows in 128; the fourth wave, which has no rows, may as well idle: no change; 14 us of
// it the join), in bf16 107 with 3 (4.3 TB/s) and 121 with 6.  6 of up to 32768 (bf16, 64 nodes, 6 heads of
// 256 on each of 4) take 435 us: 478 TFLOP/s of the products, 717 of the matrix instructions, 58 % of a large
// matrix product's rate, with LDS busy half of the time: a wave has room for 16 rows' sums, and every 16 rows
// read the whole tile.
// Four waves of 32 rows, one on a SIMD, took 637 us, without the overlap 488, where this took 455.
#include <algorithm>

#include "common.hpp"
#include "drafts.hpp"
#include "mixers_device.hpp"
#include "tree_splits.hpp"

namespace nvfp4 {
namespace {

constexpr float kNone = -3.402823466e38f;  // reference before any token: finite, so that differences are numbers
constexpr float kMost = 256.0f;             // a weight above this moves the reference
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
__device__ __forceinline__ Range range_of(const TreeArgs& a, int length) {
  const int ctx = min(max(length, 0), a.max_len);
  const int begin = a.window > 0 && a.window < ctx ? (ctx - a.window) / kTreeTile * kTreeTile : 0;
  return {ctx, begin, ctx + a.nodes - begin};
}

template <int DIM, bool FP8>
struct Shape {
  static constexpr int kRow = DIM * (FP8 ? 1 : 2);  // bytes of a cache row
  static constexpr int kLanes = kRow / 16;
  static constexpr int kLdsRow = DIM * 2;
  static constexpr int kLdsTile = 2 * kTreeTile * kLdsRow;

  // Where 16-byte piece `piece` of a row lies in LDS.  An access of 16 bytes a lane is served 16 lanes at a
  // time, of which 8 come from one run of 16 lanes and 8 from the next: here the 16 rows (keys) or pieces
  // (values) of such a set, from two neighbouring g, always fall on different banks, and so do the two rows
  // that E4M3 lanes write side by side.  (Counted: conflicts take none of the time over bf16, 6 % over E4M3; with rows
  // padded by 16 bytes instead 17 to 19 %.)
  static __device__ __forceinline__ int key_spot(int row, int piece) {
    return row * kLdsRow + (piece ^ (DIM == 64 ? row / 2 % 8 : row % 16)) * 16;
  }
  static __device__ __forceinline__ int value_spot(int row, int piece) {
    if (DIM == 64) return (row ^ row / 4 % 2) * kLdsRow + (piece ^ row / 2 % 2) * 16;
    return row * kLdsRow + (piece ^ row % 4) * 16;
  }
};

__device__ __forceinline__ uint32_t fp8_bf16(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
template <class T>
__device__ __forceinline__ T octet(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(T, make_uint4(a, b, c, d));
}

// Two bf16 values, 0 for one that is no finite number.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// A set of nodes, as two words: a shift of 64 bits by an amount in the last vector register that a wave has reads
// a wrong amount, which the compiler does not know of (with 256 registers to a wave nodes saw rows of others).
struct Nodes {
  uint32_t lo, hi;
  __device__ __forceinline__ bool none() const { return (lo | hi) == 0; }
  __device__ __forceinline__ int count() const { return __popc(lo) + __popc(hi); }
  __device__ __forceinline__ uint32_t has(int node) const {  // (mod 64)
    const uint32_t l = lo, h = hi;
    return (node & 32 ? h : l) >> (node & 31) & 1u;
  }
  __device__ __forceinline__ Nodes without_first() const {
    const uint32_t l = lo, h = hi;
    return {l & (l - 1), l ? h : h & (h - 1)};
  }
  __device__ __forceinline__ Nodes of(int lane) const { return {__shfl(lo, lane), __shfl(hi, lane)}; }
};

// Nodes on each lane's way to the context, itself included, from the lanes' parents; none for a padded node.
__device__ __forceinline__ Nodes ancestors(int nodes, int lane, int up) {
  if (lane >= nodes || up < -1 || up >= lane) up = -2;
  const uint32_t own = 1u << (lane & 31);
  Nodes seen = {lane < 32 ? own : 0, lane < 32 ? 0 : own};
  for (int s = 1; s < nodes; s *= 2) {
    const int at = max(up, 0);
    const Nodes more = seen.of(at);
    const int next = __shfl(up, at);
    if (up >= 0) seen.lo |= more.lo, seen.hi |= more.hi, up = next;
  }
  if (up != -1) seen = {0, 0};
  return seen;
}

__device__ __forceinline__ int64_t lane_value(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)x, lane), hi = __builtin_amdgcn_readlane((uint32_t)(x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// All waves of the workgroup have written to LDS what any reads from here on, and read what any
// overwrites; loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Where a row's result goes: the output, or the partial results of a split.
struct Sink {
  const TreeArgs& a;
  float* parts;
  float2* ml;
  float vg;
  int b, kvh, group, splits, split;
  bool only;
  __device__ __forceinline__ int64_t token(int row) const { return (int64_t)b * a.nodes + row / group; }
  __device__ __forceinline__ int head(int row) const { return kvh * group + row % group; }
  __device__ __forceinline__ int64_t part(int row) const { return (token(row) * a.q_heads + head(row)) * splits + split; }
};

template <int DIM, bool FP8, int NR, int RW, int KW, int MIN>
__global__ __launch_bounds__(RW* KW * 64, MIN) void attn_tree_kernel(TreeArgs a, Plan plan) {
  using Sh = Shape<DIM, FP8>;
  constexpr int ES = FP8 ? 1 : 2, PAD = DIM + 4, kRows = NR * RW * 16, kWaves = RW * KW;
  constexpr int kPieces = kTreeTile * Sh::kLanes, kMembers = RW * 64;  // of a tile's keys; lanes that load a tile
  constexpr int kLoads = (kPieces + kMembers - 1) / kMembers;          // of a lane, for keys and for values
  constexpr int kBuffers = RW > 1 ? 2 : 1;
  constexpr int kAhead = 32;                                           // turns whose pages a wave has looked up
  const nvfp4_kv_cache& c = a.cache;
  const int splits = plan.splits, group = a.q_heads / c.kv_heads;
  const int gx = c.kv_heads * plan.blocks;
  // the workgroups of one split run side by side on one XCD: the tiles come from its cache
  const uint32_t turn_xcd = blockIdx.x / 8, which = turn_xcd % gx, item = (turn_xcd / gx) * 8 + blockIdx.x % 8;
  const int kvh = which / plan.blocks, block = which % plan.blocks;
  const int b = item / splits, split = (item % splits + b / (8 / min(8, splits & -splits))) % splits;
  if (b >= a.B) return;
  const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), rw = wave % RW, kw = wave / RW;

  // What the first tile waits for starts side by side: lengths, parents, queries.
  const int length = a.lens[b];
  int parent = a.parents ? (lane < a.nodes ? a.parents[(int64_t)b * a.nodes + lane] : -2) : lane - 1;
  // rows: node * group + head, blocks of 16 to a wave
  const int all_rows = a.nodes * group, row0 = block * kRows + rw * NR * 16;
  uint4 q_read[NR][DIM / 32];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int row = min(row0 + n * 16 + r, all_rows - 1);
    const uint16_t* qp = a.q + ((int64_t)b * a.nodes + row / group) * a.ldq + (int64_t)(kvh * group + row % group) * DIM;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i) q_read[n][i] = *reinterpret_cast<const uint4*>(qp + i * 32 + g * 8);
  }

  const Range range = range_of(a, length);
  const int split_tokens = plan.tokens_of(range.span);
  const int from = range.begin + split * split_tokens, end = range.ctx + a.nodes;
  const int to = min(end, from + split_tokens);
  const bool only = split_tokens >= range.span;  // the sequence has one split: no join
  if (split > 0 && from >= end) return;

  const Nodes anc_lane = ancestors(a.nodes, lane, parent);
  const uint64_t somebody = __ballot(!anc_lane.none());
  const Nodes alive = {(uint32_t)somebody, (uint32_t)(somebody >> 32)};  // nodes that are not padded: their rows are in the cache
  const float scale = a.scale * (FP8 ? *c.k_amax / 448.0f : 1.0f) * kLog2e;
  // scores of the sign that makes the factor positive, so that the largest is the largest score
  const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
  const float factor = fmaxf(fabsf(scale), 1e-37f);
  Nodes anc[NR];
  int low[NR];  // first token of the context that the row sees
  bf16x8_t q[NR][DIM / 32];
  bool any = false;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int node = min(row0 + n * 16 + r, all_rows - 1) / group;
    anc[n] = anc_lane.of(node);
    low[n] = 0;
    any |= !anc[n].none() && row0 + n * 16 + r < all_rows;
    if (a.window > 0 && !anc[n].none()) {
      int own = anc[n].count();
      for (; own > a.window; --own) anc[n] = anc[n].without_first();  // the farthest ancestors
      low[n] = max(0, range.ctx - (a.window - own));
    }
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i) {
      const uint4 w = q_read[n][i];
      q[n][i] = octet<bf16x8_t>(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip);
    }
  }
  // tiles below hold tokens that some row's window leaves out
  const int edge = a.window > 0 ? max(0, range.ctx - max(0, a.window - a.nodes)) : 0;

  extern __shared__ float4_t dynamic_lds[];
  uint8_t* corner = reinterpret_cast<uint8_t*>(dynamic_lds) + kw * kBuffers * Sh::kLdsTile;
  float m[NR];
  float4_t sum[NR], o[NR][DIM / 16];  // sum: of the weights, the same in all four
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    m[n] = kNone, sum[n] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) o[n][i] = {0, 0, 0, 0};
  }

  // tiles from / 32 + kw + KW * turn, as many turns for all waves (barriers where waves share a tile)
  const int tile0 = from / kTreeTile + kw, tile_end = (to + kTreeTile - 1) / kTreeTile;
  const bool work = RW > 1 ? __syncthreads_or(any) : __any(any);
  const int turns = work && c.num_pages > 0 ? (tile_end - from / kTreeTile + KW - 1) / KW : 0;
  const uint8_t* kc = static_cast<const uint8_t*>(c.k) + (int64_t)kvh * c.head_stride * ES;
  const uint8_t* vc = static_cast<const uint8_t*>(c.v) + (int64_t)kvh * c.head_stride * ES;
  const int half_last = (end - 1) / 16;  // the last 16 tokens, half a tile

  // a lane's pieces of a tile: place in its half's rows, in LDS, and whether the half is the second (lanes
  // beyond the last piece load and store that one too)
  const int member = rw * 64 + lane;
  uint32_t place[kLoads], key_spot[kLoads], value_spot[kLoads];  // (of E4M3 pieces the first of two: the other is across bit 4)
  bool second[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int p = min(i * kMembers + member, kPieces - 1), row = p / Sh::kLanes, col = p % Sh::kLanes;
    place[i] = (uint32_t)(row % 16) * (uint32_t)c.token_stride * ES + col * 16;
    key_spot[i] = Sh::key_spot(row, FP8 ? 2 * col : col);
    value_spot[i] = Sh::value_spot(row, FP8 ? 2 * col : col);
    second[i] = row >= 16;
  }

  const int key_read = Sh::key_spot(r, g);
  int value_read[4];  // of tokens 4 g + j
#pragma unroll
  for (int j = 0; j < 4; ++j)
    value_read[j] = DIM == 64 ? Sh::value_spot(g * 4 + j, r / 2) + r % 2 * 8 : Sh::value_spot(g * 4 + j, r);

  // A turn's pages: places of its tile's halves in the cache, and which of them are in no page of the pool.
  struct Place {
    int64_t first, step;  // of the first half, and from there to the second
    uint32_t gone;
  };
  int64_t lane_at = 0;  // of half `lane` of the turns ahead
  uint64_t lane_gone = 0;
  auto look_up = [&](uint32_t turn) {
    if (turn % kAhead == 0) {  // (looked up again where the last turn is: the same)
      const int half = min((tile0 + ((int)turn + lane / 2) * KW) * 2 + lane % 2, half_last), token = half * 16, index = token / c.page_size;
      const int page = a.table[(int64_t)b * a.ldt + index];
      const bool gone = page < 0 || page >= c.num_pages;
      lane_gone = __ballot(gone);
      lane_at = ((int64_t)(gone ? 0 : page) * c.page_stride + (int64_t)(token - index * c.page_size) * c.token_stride) * ES;
    }
    const uint32_t at = turn % kAhead * 2;
    const int64_t first = lane_value(lane_at, at);
    return Place{first, lane_value(lane_at, at + 1) - first, (uint32_t)(lane_gone >> at) & 3u};
  };
  struct Held {
    u32x4_t x[kLoads];
  };
  auto fetch = [&](const uint8_t* from_cache, const Place& p, Held& h) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      h.x[i] = *reinterpret_cast<const u32x4_t*>(from_cache + (p.first + (second[i] ? p.step : 0) + place[i]));
  };
  auto is_masked = [&](int turn, uint32_t gone) {
    const int start = (tile0 + turn * KW) * kTreeTile;
    return start + kTreeTile > range.ctx || start < edge || gone != 0 || (KW > 1 && tile0 + turn * KW >= tile_end);
  };
  auto put_keys = [&](const Held& h, uint8_t* lds) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if constexpr (FP8) {
        uint32_t w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = fp8_bf16(h.x[i][x / 2], x % 2);
        *reinterpret_cast<uint4*>(lds + key_spot[i]) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(lds + (key_spot[i] ^ 16)) = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        *reinterpret_cast<u32x4_t*>(lds + key_spot[i]) = h.x[i];
      }
    }
  };
  uint32_t dropped = 0;  // bits of values of this lane that `put_values` took for 0 in rows that somebody sees
  auto put_values = [&](const Held& h, int turn, bool masked, uint8_t* lds) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t w[FP8 ? 8 : 4];
#pragma unroll
      for (int x = 0; x < (FP8 ? 8 : 4); ++x) {
        if constexpr (FP8)
          w[x] = fp8_bf16(h.x[i][x / 2], x % 2);
        else
          w[x] = h.x[i][x];
      }
      if (masked) {
        const int token = (tile0 + turn * KW) * kTreeTile + min(i * kMembers + member, kPieces - 1) / Sh::kLanes;
        uint32_t gone = 0;
#pragma unroll
        for (int x = 0; x < (FP8 ? 8 : 4); ++x) {
          const uint32_t kept = finite_pair(w[x]);
          gone |= w[x] ^ kept;
          w[x] = kept;
        }
        dropped |= token < range.ctx || (token < end && alive.has(token - range.ctx)) ? gone : 0;
      }
      *reinterpret_cast<uint4*>(lds + value_spot[i]) = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (FP8) *reinterpret_cast<uint4*>(lds + (value_spot[i] ^ 16)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  };

  struct Scores {
    float4_t x[NR][2];
  };
  struct Weights {
    bf16x8_t hi[NR], lo[NR];
  };
  struct Keys {
    uint4 x[DIM / 32][2];
  };
  auto read_keys = [&](const uint8_t* lds) {
    Keys k;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)  // (pieces 4 i + g: i < 4 moves them within 256 bytes)
        k.x[i][h] = *reinterpret_cast<const uint4*>(lds + (key_read ^ i % 4 * 64) + h * 16 * Sh::kLdsRow + i / 4 * 256);
    return k;
  };
  auto scores_of = [&](const Keys& k) {
    Scores s;
#pragma unroll
    for (int n = 0; n < NR; ++n) s.x[n][0] = s.x[n][1] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = k.x[i][h];
        const bf16x8_t x = octet<bf16x8_t>(w.x, w.y, w.z, w.w);
#pragma unroll
        for (int n = 0; n < NR; ++n) s.x[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, q[n][i], s.x[n][h], 0, 0, 0);
      }
    return s;
  };
  auto mask = [&](Scores& s, int turn, uint32_t gone) {
    const int start = (tile0 + turn * KW) * kTreeTile;
    if (tile0 + turn * KW >= tile_end) gone = 3;  // the last turn may have fewer tiles than groups
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = start + e / 4 * 16 + g * 4 + e % 4, drafted = t - range.ctx;
        const uint32_t in_tree = drafted < 64 ? anc[n].has(drafted) : 0u;
        const uint32_t in_context = t >= low[n] ? 1u : 0u;
        const uint32_t seen = (drafted < 0 ? in_context : in_tree) & ~(gone >> (e / 4));
        s.x[n][e / 4][e % 4] = seen & 1u ? s.x[n][e / 4][e % 4] : -INFINITY;
      }
  };
  // One score's weight under the row's reference.
  auto weigh = [&](const Scores& s, float (&p)[NR][8]) {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) p[n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s.x[n][e / 4][e % 4], factor, -m[n]));
  };
  auto largest = [](const float (&x)[8]) {
    return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  };
  // Weights for the product with the values; the references move where one of them is too large.
  auto settle = [&](const Scores& s, float (&p)[NR][8]) {
    float most = largest(p[0]);
#pragma unroll
    for (int n = 1; n < NR; ++n) most = fmaxf(most, largest(p[n]));
    if (__any(most > kMost)) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s.x[n][e / 4][e % 4];
        float top = largest(x) * factor;
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m[n]);
        const float keep = __builtin_amdgcn_exp2f(m[n] - top);
        m[n] = top;
        sum[n] *= keep;
#pragma unroll
        for (int i = 0; i < DIM / 16; ++i) o[n][i] *= keep;
      }
      weigh(s, p);
    }
    Weights w;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      uint32_t hw[4], lw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = p[n][2 * e], y = p[n][2 * e + 1];
        hw[e] = bf16_pair(x, y);
        lw[e] = bf16_pair(x - __uint_as_float(hw[e] << 16), y - __uint_as_float(hw[e] & 0xFFFF0000u));
      }
      w.hi[n] = octet<bf16x8_t>(hw[0], hw[1], hw[2], hw[3]);
      w.lo[n] = octet<bf16x8_t>(lw[0], lw[1], lw[2], lw[3]);
    }
    return w;
  };
  // values: tokens 16 s + 4 g + j in runs of 16 bytes at most
  constexpr int kRun = DIM < 128 ? DIM / 32 : 4, kRuns = DIM / 32 / kRun;  // dwords of a run; runs of a row
  struct Run {
    uint32_t x[8][kRun];
  };
  auto read_run = [&](const uint8_t* lds, int u) {
    Run v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* p = lds + value_read[e % 4] + e / 4 * 16 * Sh::kLdsRow + u * 256;
      if constexpr (kRun == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v.x[e][0] = x.x, v.x[e][1] = x.y;
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v.x[e][0] = x.x, v.x[e][1] = x.y, v.x[e][2] = x.z, v.x[e][3] = x.w;
      }
    }
    return v;
  };
  // The values, whose first run has been read.
  auto add_values = [&](const Weights& w, const Run& first, const uint8_t* lds) {
    auto add = [&](bf16x8_t v, int n, float4_t& to) {
      to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w.lo[n], to, 0, 0, 0);
      to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w.hi[n], to, 0, 0, 0);
    };
    constexpr uint32_t kOnes = 0x3F803F80u;
#pragma unroll
    for (int n = 0; n < NR; ++n) add(octet<bf16x8_t>(kOnes, kOnes, kOnes, kOnes), n, sum[n]);
#pragma unroll
    for (int u = 0; u < kRuns; ++u) {
      const Run v = u == 0 ? first : read_run(lds, u);
#pragma unroll
      for (int x = 0; x < kRun; ++x) {
        const bf16x8_t even = octet<bf16x8_t>(low_halves(v.x[0][x], v.x[1][x]), low_halves(v.x[2][x], v.x[3][x]),
                                              low_halves(v.x[4][x], v.x[5][x]), low_halves(v.x[6][x], v.x[7][x]));
        const bf16x8_t odd = octet<bf16x8_t>(high_halves(v.x[0][x], v.x[1][x]), high_halves(v.x[2][x], v.x[3][x]),
                                             high_halves(v.x[4][x], v.x[5][x]), high_halves(v.x[6][x], v.x[7][x]));
        const int i = (u * kRun + x) * 2;
#pragma unroll
        for (int n = 0; n < NR; ++n) add(even, n, o[n][i]), add(odd, n, o[n][i + 1]);
      }
    }
  };

  // (Loads and stores below are unconditional, of the last turn's tile again behind the end: for a load that
  // may not have been issued the compiler waits with all others.)
  const int last = turns - 1;
  if constexpr (RW == 1) {  // each wave alone, with a tile in LDS and the next on its way
    uint8_t* values = corner + kTreeTile * Sh::kLdsRow;
    Held k, v;
    uint32_t gone = 0;
    auto start_turn = [&](int t) {
      const Place p = look_up(t);
      fetch(kc, p, k);
      fetch(vc, p, v);
      gone = p.gone;
    };
    if (turns > 0) start_turn(0);
    for (int t = 0; t < turns; ++t) {
      const uint32_t gone_now = gone;
      const bool masked = is_masked(t, gone_now);
      put_keys(k, corner);
      put_values(v, t, masked, values);
      wave_lds_fence();
      start_turn(min(t + 1, last));
      Scores s = scores_of(read_keys(corner));
      const Run v0 = read_run(values, 0);
      if (masked) mask(s, t, gone_now);
      float p[NR][8];
      weigh(s, p);
      const Weights w = settle(s, p);
      add_values(w, v0, values);
      wave_lds_fence();
    }
  } else if (turns > 0) {
    // Turn t multiplies the values of tile t while the scores of tile t + 1 are formed: the matrix units have
    // these to do while the vector units weigh.  Two buffers of keys and two of values in LDS: in turn t the
    // keys of t + 2 and the values of t + 1 are put there, and the next ones fetched.  (A second set of them on
    // its way changed nothing.)
    uint8_t* keys[2] = {corner, corner + kTreeTile * Sh::kLdsRow};
    uint8_t* values[2] = {corner + 2 * kTreeTile * Sh::kLdsRow, corner + 3 * kTreeTile * Sh::kLdsRow};
    Held k, v;
    uint32_t gone = 0;  // two bits a turn, the latest that was looked up in the lowest
    Place ahead;        // of the turn whose keys were fetched last
    auto fetch_keys = [&](int t) {
      ahead = look_up(min(t, last));
      gone = gone << 2 | ahead.gone;
      fetch(kc, ahead, k);
    };
    fetch_keys(0);
    fetch(vc, ahead, v);
    put_keys(k, keys[0]);
    put_values(v, 0, is_masked(0, gone & 3u), values[0]);
    fetch_keys(1);
    fetch(vc, ahead, v);
    lds_barrier();
    Scores s = scores_of(read_keys(keys[0]));
    put_keys(k, keys[1]);
    fetch_keys(2);
    lds_barrier();
    // Turn t; `odd`: t % 2, the same for its buffers.  In registers: the keys of t + 2, the values of t + 1.
    auto step = [&](int t, int odd) {
      const uint32_t gone_now = gone >> 4 & 3u, gone_next = gone >> 2 & 3u;
      const Keys read = read_keys(keys[odd ^ 1]);
      put_keys(k, keys[odd]);
      put_values(v, min(t + 1, last), is_masked(min(t + 1, last), gone_next), values[odd ^ 1]);
      fetch(vc, ahead, v);  // of turn t + 2
      fetch_keys(t + 3);
      if (is_masked(t, gone_now)) mask(s, t, gone_now);
      float p[NR][8];
      weigh(s, p);
      const Scores next = scores_of(read);
      const Run v0 = read_run(values[odd], 0);
      __builtin_amdgcn_sched_barrier(0);  // on its way while the weights settle
      const Weights w = settle(s, p);
      add_values(w, v0, values[odd]);
      s = next;
      lds_barrier();
    };
    for (int t = 0; t < turns; t += 2) {
      step(t, 0);
      if (t + 1 < turns) step(t + 1, 1);
    }
  }

  // element of the row that output tile i holds in row 4 g + j: value rows are read in runs of 16 bytes at most
  constexpr int kEach = DIM == 256 ? 8 : DIM / 16;

  // Dropped values reach the rows that see them: their tiles are looked through again, a token at a time.
  if (RW > 1 ? __syncthreads_or(dropped != 0) : __any(dropped != 0)) {
#pragma unroll 1
    for (int t = 0; t < turns; ++t) {
      const Place p = look_up(t);
      if (!is_masked(t, p.gone) || tile0 + t * KW >= tile_end) continue;
      const int start = (tile0 + t * KW) * kTreeTile;
#pragma unroll 1
      for (int x = 0; x < min(kTreeTile, end - start); ++x) {
        if (p.gone >> (x / 16) & 1u) continue;
        const int drafted = start + x - range.ctx;
        bool sees[NR], one = false;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          sees[n] = !anc[n].none() && (drafted < 0 ? start + x >= low[n] : anc[n].has(drafted) != 0);
          one |= sees[n];
        }
        if (!__any(one)) continue;
        const uint8_t* row = vc + p.first + (x < 16 ? 0 : p.step) + (int64_t)(x % 16) * c.token_stride * ES;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < DIM / 16; ++i) {
            const int at = i / kEach * 128 + (g * 4 + j) * kEach + i % kEach;
            const uint32_t code = FP8 ? row[at] : reinterpret_cast<const uint16_t*>(row)[at];
            const float value = FP8 ? __builtin_nanf("") : __uint_as_float(code << 16);
            const uint32_t exponent = FP8 ? 0x7Fu : 0x7F80u;
            if ((code & exponent) == exponent) {
#pragma unroll
              for (int n = 0; n < NR; ++n) o[n][i][j] += sees[n] ? value : 0.0f;
            }
          }
      }
    }
  }

  float l[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    l[n] = sum[n][0];
    if (anc[n].none()) {  // a padded node: the tiles of the context have no mask
      m[n] = kNone, l[n] = 0;
#pragma unroll
      for (int i = 0; i < DIM / 16; ++i) o[n][i] = {0, 0, 0, 0};
    }
  }
  float* parts = static_cast<float*>(a.workspace);
  const Sink sink = {a, parts, reinterpret_cast<float2*>(parts + (int64_t)a.B * a.nodes * a.q_heads * splits * DIM),
                     FP8 ? *c.v_amax / 448.0f : 1.0f, b, kvh, group, splits, split, only};
  if constexpr (KW == 1) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = row0 + n * 16 + r;
      if (row >= all_rows) continue;
      const float by = only ? (l[n] == 0 ? 0.0f : sink.vg / l[n]) : 1.0f;
      const int64_t token = sink.token(row), part = sink.part(row);
      const int head = sink.head(row);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < DIM / 16; i += kEach) {
          const int at = i / kEach * 128 + (g * 4 + j) * kEach;
          if (only) {
            uint32_t w[kEach / 2];
#pragma unroll
            for (int x = 0; x < kEach / 2; ++x) w[x] = bf16_pair(o[n][i + 2 * x][j] * by, o[n][i + 2 * x + 1][j] * by);
            uint16_t* to_out = a.out + token * a.ldo + (int64_t)head * DIM + at;
            if constexpr (kEach == 8)
              *reinterpret_cast<uint4*>(to_out) = make_uint4(w[0], w[1], w[2], w[3]);
            else
              *reinterpret_cast<uint2*>(to_out) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int x = 0; x < kEach; x += 4)
              *reinterpret_cast<float4_t*>(parts + part * DIM + at + x) =
                  float4_t{o[n][i + x][j], o[n][i + x + 1][j], o[n][i + x + 2][j], o[n][i + x + 3][j]};
          }
        }
      if (g == 0) {
        if (!only)
          sink.ml[part] = make_float2(m[n], l[n]);
        else if (a.lse)
          a.lse[token * a.q_heads + head] = l[n] == 0 ? -INFINITY : m[n] * kLn2 + logf(l[n]);
      }
    }
  } else {
    // the groups' results, joined in LDS
    __shared__ float ms[kWaves][NR * 16], ls[kWaves][NR * 16];
    float* os = reinterpret_cast<float*>(dynamic_lds);  // [group][kRows][PAD], over the tiles
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if (g == 0) ms[wave][n * 16 + r] = m[n], ls[wave][n * 16 + r] = l[n];
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
    const int mine = min(kRows, all_rows - block * kRows);
    for (int e = threadIdx.x * 4; e < mine * DIM; e += kWaves * 64 * 4) {
      const int row = e / DIM, d = e % DIM, w0 = row / (NR * 16), in = row % (NR * 16);
      float top = kNone, total = 0;
#pragma unroll
      for (int w = 0; w < KW; ++w) top = fmaxf(top, ms[w * RW + w0][in]);
      float4_t x = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float f = __builtin_amdgcn_exp2f(ms[w * RW + w0][in] - top);
        total += ls[w * RW + w0][in] * f;
        x += *reinterpret_cast<const float4_t*>(os + (w * kRows + row) * PAD + d) * f;
      }
      const int64_t token = sink.token(block * kRows + row), part = sink.part(block * kRows + row);
      const int head = sink.head(block * kRows + row);
      if (only) {
        const float4_t y = x * (total == 0 ? 0.0f : sink.vg / total);
        *reinterpret_cast<uint2*>(a.out + token * a.ldo + (int64_t)head * DIM + d) = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
        if (a.lse && d == 0) a.lse[token * a.q_heads + head] = total == 0 ? -INFINITY : top * kLn2 + logf(total);
      } else {
        *reinterpret_cast<float4_t*>(parts + part * DIM + d) = x;
        if (d == 0) sink.ml[part] = make_float2(top, total);
      }
    }
  }
}

// Joins the splits of the rows: each counts 2^(its m - the largest m), in a fixed order.  A row has DIM / 4 lanes
// side by side, which take kJoin splits at a time, or, for fewer rows of more splits, 4 or 16 such sets of lanes.
// Attention and join, us, with one set, four and sixteen (E4M3, heads of 128; *: bf16, 256):
//   rows x splits   200 x 7   200 x 12   640 x 12   40 x 61   640 x 188   1000 x 61   768* x 61   1280 x 23   1920 x 47   2560 x 23
//   one             14.8      15.8       21.2       28.8      150         55.1        89.8        43.0        74.0        51.6
//   four            14.8      15.3       20.9       27.1      148         54.4        88.4        42.4        72.7        51.4
//   sixteen         14.9      15.3       22.3       24.3      144         53.2        92.3        44.6        76.4        57.7
// (and 48 sequences of 16 nodes and 40 heads in up to four splits, 30720 rows: 14 us of join with one, 24 with four).
constexpr int kJoin = 8;
constexpr int64_t kFewRows = 2048, kFewColumns = 1 << 17;

template <int DIM, bool FP8>
__device__ __forceinline__ void store_row(const TreeArgs& a, int64_t row, int d, float4_t x, float m, float sum) {
  const int64_t token = row / a.q_heads;
  const int head = (int)(row - token * a.q_heads);
  x = x * (sum == 0 ? 0.0f : (FP8 ? *a.cache.v_amax / 448.0f : 1.0f) / sum);
  *reinterpret_cast<uint2*>(a.out + token * a.ldo + (int64_t)head * DIM + d) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
  if (a.lse && d == 0) a.lse[row] = sum == 0 ? -INFINITY : m * kLn2 + logf(sum);
}

template <int DIM, bool FP8>
__global__ __launch_bounds__(256) void tree_join_kernel(TreeArgs a, Plan plan) {
  constexpr int kLanes = DIM / 4;
  const int splits = plan.splits, d = threadIdx.x % kLanes * 4;
  const int64_t rows = (int64_t)a.B * a.nodes * a.q_heads;
  const int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  if (row >= rows) return;
  const Range range = range_of(a, a.lens[(uint32_t)row / (uint32_t)(a.q_heads * a.nodes)]);
  const int split_tokens = plan.tokens_of(range.span), used = (range.span + split_tokens - 1) / split_tokens;
  if (used <= 1) return;
  const float* parts = static_cast<const float*>(a.workspace);
  const float2* ml = reinterpret_cast<const float2*>(parts + rows * splits * DIM) + row * splits;
  const float* x_row = parts + row * splits * DIM + d;
  float m = kNone, sum = 0;
  float4_t x = {0, 0, 0, 0};
  for (int s0 = 0; s0 < used; s0 += kJoin) {
    float2 w[kJoin];
    float4_t v[kJoin];
#pragma unroll
    for (int s = 0; s < kJoin; ++s) {  // on their way side by side
      const int at = min(s0 + s, used - 1);
      w[s] = ml[at];
      v[s] = *reinterpret_cast<const float4_t*>(x_row + (int64_t)at * DIM);
    }
    float top = m;
#pragma unroll
    for (int s = 0; s < kJoin; ++s) top = fmaxf(top, w[s].x);
    const float keep = __builtin_amdgcn_exp2f(m - top);
    m = top;
    sum *= keep, x *= keep;
#pragma unroll
    for (int s = 0; s < kJoin; ++s) {
      const float f = s0 + s < used ? __builtin_amdgcn_exp2f(w[s].x - m) : 0.0f;
      sum += w[s].y * f;
      x += v[s] * f;
    }
  }
  store_row<DIM, FP8>(a, row, d, x, m, sum);
}

template <int DIM, bool FP8, int kGroups>
__global__ __launch_bounds__(DIM / 4 * kGroups) void tree_join_many_kernel(TreeArgs a, Plan plan) {
  constexpr int kLanes = DIM / 4;
  const int splits = plan.splits;
  const int64_t row = blockIdx.x;
  const int d = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const Range range = range_of(a, a.lens[row / (a.q_heads * a.nodes)]);
  const int split_tokens = plan.tokens_of(range.span), used = (range.span + split_tokens - 1) / split_tokens;
  if (used <= 1) return;
  const float* parts = static_cast<const float*>(a.workspace);
  const float2* ml = reinterpret_cast<const float2*>(parts + (int64_t)a.B * a.nodes * a.q_heads * splits * DIM) + row * splits;
  const float* x_row = parts + row * splits * DIM + d * 4;
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
  store_row<DIM, FP8>(a, row, d * 4, x, top, sum);
}

// Rows of a workgroup, by the rows of a key-value head.  (80 rows in 96 of three waves took 6 % longer than in
// 128 of four: two such workgroups leave two SIMDs of a CU with one wave.)
int wg_rows(int64_t rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128)); }

Plan tree_plan(int64_t B, int nodes, int q_heads, int kv_heads, int head_dim, int64_t max_len, int64_t window) {
  const int64_t rows = (int64_t)nodes * (q_heads / kv_heads), per = wg_rows(rows);
  const int64_t blocks = (rows + per - 1) / per, each = B * kv_heads * blocks;
  const Splits s = tree_splits(each, max_len, nodes, window);
  return {(int)each, (int)blocks, s.count, s.tokens, (int)tree_span(max_len, nodes, window)};
}

template <int DIM, bool FP8, int NR, int RW, int KW, int MIN>
hipError_t launch_rows(const TreeArgs& a, const Plan& plan, hipStream_t stream) {
  constexpr size_t tiles = (size_t)KW * (RW > 1 ? 2 : 1) * Shape<DIM, FP8>::kLdsTile;
  constexpr size_t lds = KW == 1 ? tiles : std::max<size_t>(tiles, (size_t)KW * NR * RW * 16 * (DIM + 4) * sizeof(float));
  hipError_t e = hipSuccess;
  if (lds > 48 * 1024)  // the same for every call, from whatever thread
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_tree_kernel<DIM, FP8, NR, RW, KW, MIN>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((int64_t)a.cache.kv_heads * plan.blocks * (((int64_t)a.B * plan.splits + 7) / 8 * 8)));
  attn_tree_kernel<DIM, FP8, NR, RW, KW, MIN><<<grid, RW * KW * 64, lds, stream>>>(a, plan);
  return hipGetLastError();
}

template <int DIM, bool FP8>
hipError_t launch_dim(const TreeArgs& a, hipStream_t stream) {
  const Plan plan = tree_plan(a.B, a.nodes, a.q_heads, a.cache.kv_heads, DIM, a.max_len, a.window);
  hipError_t e;
  const int rows = wg_rows((int64_t)a.nodes * (a.q_heads / a.cache.kv_heads));
  // Few rows: groups of waves that take tiles in turn.  More: waves that share a tile, two blocks of 16 rows to
  // each where the accumulators leave room (heads of 256: one).  What spills is not taken: two blocks to each of
  // four such groups took 191 us for 48 sequences, 30 rows, in bf16, two waves with one block in two groups 120
  // (E4M3: 72 and 75, one sequence of 32768 29.7 and 27.1); heads of 256 have one wave on a SIMD there, 148 us
  // against 228 for 6 x 32768.
  if constexpr (DIM == 256) {
    e = rows == 16   ? launch_rows<DIM, FP8, 1, 1, 4, 1>(a, plan, stream)
        : rows == 32 ? launch_rows<DIM, FP8, 1, 2, 2, 1>(a, plan, stream)
        : rows == 64 ? launch_rows<DIM, FP8, 1, 4, 1, 2>(a, plan, stream)
                     : launch_rows<DIM, FP8, 1, 8, 1, 2>(a, plan, stream);
  } else {
    e = rows == 16   ? launch_rows<DIM, FP8, 1, 1, 4, 2>(a, plan, stream)
        : rows == 32 ? launch_rows<DIM, FP8, 1, 2, 2, 2>(a, plan, stream)
        : rows == 64 ? launch_rows<DIM, FP8, 1, 4, 1, 2>(a, plan, stream)
                     : launch_rows<DIM, FP8, 2, 4, 1, 2>(a, plan, stream);
  }
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t all = (int64_t)a.B * a.nodes * a.q_heads;
  if (plan.splits <= kJoin || all >= kFewRows)
    tree_join_kernel<DIM, FP8><<<dim3((unsigned)((all + 1024 / DIM - 1) / (1024 / DIM))), 256, 0, stream>>>(a, plan);
  else if (plan.splits <= 16 || all * DIM > kFewColumns)
    tree_join_many_kernel<DIM, FP8, 4><<<dim3((unsigned)all), DIM, 0, stream>>>(a, plan);
  else
    tree_join_many_kernel<DIM, FP8, 16><<<dim3((unsigned)all), DIM * 4, 0, stream>>>(a, plan);
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

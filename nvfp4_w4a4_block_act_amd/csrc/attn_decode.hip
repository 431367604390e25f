// Attention of one new token over the paged key-value cache.
//
// One pass over the cached tokens with a running reference m and sum l of the
// softmax (scores in units of log 2): tokens enter as 2^(s - m), and when a score
// exceeds m by more than kSlack, m moves up and the sums so far are scaled.  m
// need not be the maximum itself: sums and weights are binary32, whose range
// holds 2^kSlack with ease, and most tiles then need no exchange between lanes.
//
// Layout.  A wave takes tiles of 16 tokens (a page holds whole tiles) for up to 16
// query heads that share a key-value head.  Lanes load whole rows side by side, 16
// bytes each -- a load in operand order, 16 rows side by side, costs the vector cache
// one access a lane, four times as many (67 sequences of up to 4099: 14 % more time,
// hints below included) -- and the tile passes through a corner of LDS that only its wave uses:
//  * scores: S^T = K Q^T (16 x 16 x 32, bf16): lane (r, g) = (lane % 16, lane / 16)
//    takes 16-byte pieces of token r's key row; which elements of the row a step
//    multiplies is free as long as q is taken in the same order;
//  * S^T leaves token 4 g + j of head r in register j of lane (r, g), which is
//    where P^T must be for O^T = V^T P^T (16 x 16 x 16): the weights need no move;
//  * V^T: lane (c, g) takes its head_dim / 16 elements of the value rows of tokens
//    4 g .. 4 g + 3, and the transposition is four rows' worth of byte permutes within
//    the lane; output tile i then holds element i of every lane's run.
// A weight enters as the sum of two bf16 values (16 significant bits, two matrix
// instructions), so that its rounding (2^-17) is far below that of the output.
// E4M3 codes widen to bf16 exactly; k's scale goes into the scores' factor, v's
// into the output.  Loads of the next tile are in flight while one is computed.
//
// The tokens of a sequence are split over workgroups of four waves (wave w takes
// tiles w, w + 4, ...), joined through LDS, and over splits, whose partial results
// a second kernel joins in a fixed order.
//
// Bound by memory: each key and value once.  67 sequences of up to 4099 (350 MB of E4M3,
// 8 heads of 128) take 71 us, 4.9 TB/s; 6 of up to 32768 (541 MB of bf16, 4 heads of 256)
// 100 us, 5.4 TB/s; one of 517 tokens 8.8 us, of which the kernel is 7.3: five tiles one
// after the other in each of eight waves.  Bare reads of as many bytes take 51 to 56 and
// 78 us; rows in scattered places, two streams a workgroup, account for most of the rest,
// and more tiles or waves in flight made it slower.  More than 16 query heads of a key-value
// head read its tiles once for each 16: 64 of up to 4096 with 24 heads on each of two (82 MB)
// fetch 99 MB, the second reading mostly from the caches, and take 35 us, 2.3 TB/s, bound by
// the work on the tiles.  Rows of 64 bytes (16 heads of 64, E4M3, 322 MB): 77 us, 4.2 TB/s.
#include <algorithm>

#include "attn_splits.hpp"
#include "common.hpp"
#include "mixers.hpp"
#include "mixers_device.hpp"

namespace nvfp4 {

constexpr float kNone = -3.402823466e38f;  // reference before any token: finite, so that differences are numbers
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// How a launch splits its sequences, as the kernels get it (attn_splits.hpp).
struct Plan {
  int rows, splits, tokens, bound;
  // a sequence's own tokens of a split; a single one covers whatever there is
  __device__ __forceinline__ int tokens_of(int len, int window) const {
    return splits == 1 ? tokens : attn_split_tokens(rows, tokens, bound, (int)attn_span(len, window));
  }
};
static Plan attn_plan(int64_t B, int q_heads, int kv_heads, int64_t max_len, int64_t window) {
  const int64_t rows = B * kv_heads * ((q_heads / kv_heads + 15) / 16);
  const Splits s = attn_splits(rows, max_len, window);
  return {(int)rows, s.count, s.tokens, (int)attn_span(max_len, window)};
}

// 16 tokens' keys and values on their way: rows in pieces of 16 bytes, lanes side by side
// along a row.
template <int DIM, bool FP8>
struct Tile {
  static constexpr int kRow = DIM * (FP8 ? 1 : 2);          // bytes
  static constexpr int kLanes = kRow / 16;                  // of a row
  static constexpr int kLoads = kLanes / 4;                 // of a lane, for keys and for values
  static constexpr int kLdsRow = kRow + 16;                 // 16 rows' pieces fall on different banks
  static constexpr int kLdsBytes = 2 * 16 * kLdsRow;
  u32x4_t k[kLoads], v[kLoads];
};

// A row of whole cache lines is read once and hinted so (67 x 4099 of 128 bytes take 8 % more
// without, 6 x 32768 of 512 4 %); rows of 64 bytes share lines with the next head's, which the
// hint would drop (14 % more with it).
template <int ROW>
__device__ __forceinline__ u32x4_t load_piece(const uint8_t* p) {
  if constexpr (ROW >= 128) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  return *reinterpret_cast<const u32x4_t*>(p);
}

// k, v: the tile's first row; offset: the lane's piece of it; step: bytes between a lane's rows.
template <int DIM, bool FP8>
__device__ __forceinline__ void load_tile(Tile<DIM, FP8>& t, const uint8_t* k, const uint8_t* v, uint32_t offset,
                                          uint32_t step) {
#pragma unroll
  for (int i = 0; i < Tile<DIM, FP8>::kLoads; ++i) t.k[i] = load_piece<Tile<DIM, FP8>::kRow>(k + (offset + i * step));
#pragma unroll
  for (int i = 0; i < Tile<DIM, FP8>::kLoads; ++i) t.v[i] = load_piece<Tile<DIM, FP8>::kRow>(v + (offset + i * step));
}

// The tile into the wave's corner of LDS, keys then values.
template <int DIM, bool FP8>
__device__ __forceinline__ void put_tile(const Tile<DIM, FP8>& t, uint8_t* lds) {
  using Ti = Tile<DIM, FP8>;
  const int lane = threadIdx.x % 64;
  uint8_t* to = lds + lane / Ti::kLanes * Ti::kLdsRow + lane % Ti::kLanes * 16;
#pragma unroll
  for (int i = 0; i < Ti::kLoads; ++i) {
    *reinterpret_cast<u32x4_t*>(to + i * (64 / Ti::kLanes) * Ti::kLdsRow) = t.k[i];
    *reinterpret_cast<u32x4_t*>(to + (16 + i * (64 / Ti::kLanes)) * Ti::kLdsRow) = t.v[i];
  }
}

__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

__device__ __forceinline__ bf16x8_t octet(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(a, b, c, d));
}

__device__ __forceinline__ void store_out(uint16_t* to, float4_t x) {
  *reinterpret_cast<uint2*>(to) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
}

struct Running {
  float m, l;  // of head lane % 16; l: this lane's tokens only
};

// One tile into the running softmax and the outputs.  first, last: tokens of the
// tile that count.
template <int DIM, bool FP8>
__device__ __forceinline__ void take_tile(const uint8_t* lds, const bf16x8_t (&q)[DIM / 32], float factor, int first,
                                          int last, Running& run, float4_t (&o)[DIM / 16]) {
  using Ti = Tile<DIM, FP8>;
  constexpr int kValues = Ti::kRow / 64;  // dwords of a lane's run of a value row
  const int r = threadIdx.x % 16, g = (threadIdx.x % 64) / 16;
  float4_t s = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Ti::kRow / 64; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(lds + r * Ti::kLdsRow + i * 64 + g * 16);
    if constexpr (FP8) {
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          octet(fp8_pair(w.x, false), fp8_pair(w.x, true), fp8_pair(w.y, false), fp8_pair(w.y, true)), q[2 * i], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          octet(fp8_pair(w.z, false), fp8_pair(w.z, true), fp8_pair(w.w, false), fp8_pair(w.w, true)), q[2 * i + 1], s, 0, 0,
          0);
    } else {
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(octet(w.x, w.y, w.z, w.w), q[i], s, 0, 0, 0);
    }
  }
  uint32_t v[4][kValues];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint8_t* p = lds + (16 + g * 4 + j) * Ti::kLdsRow + (Ti::kRow < 256 ? Ti::kRow / 16 : 16) * r;
    if constexpr (kValues == 1) {
      v[j][0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kValues == 2) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[j][0] = w.x, v[j][1] = w.y;
    } else {
#pragma unroll
      for (int h = 0; h < kValues / 4; ++h) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + h * 256);
        v[j][4 * h] = w.x, v[j][4 * h + 1] = w.y, v[j][4 * h + 2] = w.z, v[j][4 * h + 3] = w.w;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] *= factor;
  if (first > 0 || last < 16) {  // uniform: the tiles at either end
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (g * 4 + j < first || g * 4 + j >= last) {
        s[j] = -INFINITY;
#pragma unroll
        for (int x = 0; x < kValues; ++x) v[j][x] = 0;  // whatever the row holds, 0 times it is 0
      }
    }
  }
  float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
  if (__any(top > run.m + kSlack)) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), run.m);
    const float keep = __builtin_amdgcn_exp2f(run.m - top);
    run.m = top;
    run.l *= keep;
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) o[i] *= keep;
  }
  float p[4], rest[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p[j] = __builtin_amdgcn_exp2f(s[j] - run.m);
    run.l += p[j];
  }
  const uint32_t h01 = bf16_pair(p[0], p[1]), h23 = bf16_pair(p[2], p[3]);
  rest[0] = p[0] - __uint_as_float(h01 << 16), rest[1] = p[1] - __uint_as_float(h01 & 0xFFFF0000u);
  rest[2] = p[2] - __uint_as_float(h23 << 16), rest[3] = p[3] - __uint_as_float(h23 & 0xFFFF0000u);
  const short4_t hi = __builtin_bit_cast(short4_t, make_uint2(h01, h23));
  const short4_t lo = __builtin_bit_cast(short4_t, make_uint2(bf16_pair(rest[0], rest[1]), bf16_pair(rest[2], rest[3])));
  auto product = [&](int i, uint32_t v01, uint32_t v23) {
    const short4_t x = __builtin_bit_cast(short4_t, make_uint2(v01, v23));
    o[i] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(x, lo, o[i], 0, 0, 0);
    o[i] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(x, hi, o[i], 0, 0, 0);
  };
#pragma unroll
  for (int x = 0; x < kValues; ++x) {
    if constexpr (FP8) {
      uint32_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = fp8_pair(v[j][x], false), b[j] = fp8_pair(v[j][x], true);
      product(4 * x, low_halves(a[0], a[1]), low_halves(a[2], a[3]));
      product(4 * x + 1, high_halves(a[0], a[1]), high_halves(a[2], a[3]));
      product(4 * x + 2, low_halves(b[0], b[1]), low_halves(b[2], b[3]));
      product(4 * x + 3, high_halves(b[0], b[1]), high_halves(b[2], b[3]));
    } else {
      product(2 * x, low_halves(v[0][x], v[1][x]), low_halves(v[2][x], v[3][x]));
      product(2 * x + 1, high_halves(v[0][x], v[1][x]), high_halves(v[2][x], v[3][x]));
    }
  }
}

// Element of the head that output tile i holds in row c: value rows are read in
// runs of 16 bytes at most, 16 lanes beside each other.
template <int DIM, bool FP8>
__device__ __forceinline__ int out_element(int c, int i) {
  if constexpr (!FP8 && DIM == 256) return (i / 8) * 128 + c * 8 + i % 8;
  return c * (DIM / 16) + i;
}

// Partial results of a split: per (sequence, query head, split) the sums, then m and l.
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, int b, int head, int splits, int s) {
  return ((int64_t)b * a.q_heads + head) * splits + s;
}

template <int DIM, bool FP8, int kWaves>
__global__ __launch_bounds__(kWaves * 64, 2) void attn_decode_kernel(AttnArgs a, Plan plan) {
  constexpr int ES = FP8 ? 1 : 2, PAD = DIM + 4;
  const int splits = plan.splits;
  const int group = a.q_heads / a.cache.kv_heads, per = (group + 15) / 16;
  const int gx = a.cache.kv_heads * per;
  const uint32_t xcd_turn = blockIdx.x / 8, which = xcd_turn % gx, item = (xcd_turn / gx) * 8 + blockIdx.x % 8;
  const int kvh = which / per, head0 = kvh * group + (which % per) * 16;
  const int heads = min(16, (kvh + 1) * group - head0);
  // The later splits of shorter sequences are empty, so each XCD has to get all of them
  // alike: where their number and eight have a factor in common, they move on by one each
  // time the pattern would repeat (16 sequences of up to 8192 in bf16: 10 % more time without).
  const int b = item / splits, split = (item % splits + b / (8 / min(8, splits & -splits))) % splits;
  if (b >= a.B) return;
  const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const nvfp4_kv_cache& c = a.cache;

  const int len = min(max(a.lens[b], 0), a.max_len);
  const int begin = a.window > 0 ? max(0, len - a.window) : 0;
  const int first_tile = begin / 16, split_tokens = plan.tokens_of(len, a.window);
  // this split's tokens, from the tile that `begin` lies in
  const int from = first_tile * 16 + split * split_tokens;
  const int to = min(len, from + split_tokens);
  const bool only = first_tile * 16 + split_tokens >= len;  // the sequence has one split: no join
  if (split > 0 && from >= len) return;

  bf16x8_t q[DIM / 32];
  {
    const uint16_t* qp = a.q + (int64_t)b * a.ldq + (int64_t)(head0 + min(r, heads - 1)) * DIM;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i)
      q[i] = *reinterpret_cast<const bf16x8_t*>(qp + (FP8 ? (i / 2) * 64 + g * 16 + (i % 2) * 8 : i * 32 + g * 8));
  }
  const float factor = a.scale * (FP8 ? *c.k_amax / 448.0f : 1.0f) * kLog2e;
  const uint8_t* kc = static_cast<const uint8_t*>(c.k) + (int64_t)kvh * c.head_stride * ES;
  const uint8_t* vc = static_cast<const uint8_t*>(c.v) + (int64_t)kvh * c.head_stride * ES;
  using Ti = Tile<DIM, FP8>;
  const uint32_t row = (uint32_t)c.token_stride * ES;
  const uint32_t offset = lane / Ti::kLanes * row + lane % Ti::kLanes * 16, step = 64 / Ti::kLanes * row;
  const int tiles_per_page = c.page_size / 16;

  extern __shared__ float4_t dynamic_lds[];
  uint8_t* corner = reinterpret_cast<uint8_t*>(dynamic_lds) + wave * Ti::kLdsBytes;  // the wave's own, for one tile
  Running run = {kNone, 0};
  float4_t o[DIM / 16];
#pragma unroll
  for (int i = 0; i < DIM / 16; ++i) o[i] = {0, 0, 0, 0};

  // tiles of this wave: from / 16 + wave + kWaves * n
  const int tile0 = from / 16 + wave, tile_end = (to + 15) / 16;
  const int mine = tile0 < tile_end && c.num_pages > 0 ? (tile_end - tile0 + kWaves - 1) / kWaves : 0;
  for (int n0 = 0; n0 < mine; n0 += 64) {
    // page and place in it of 64 tiles ahead, one in each lane
    const int ahead = min(n0 + lane, mine - 1) * kWaves + tile0;
    const int page_index = ahead / tiles_per_page;
    const int page = a.table[(int64_t)b * a.ldt + page_index];
    const int inside = ahead - page_index * tiles_per_page;
    const int count = min(64, mine - n0);
    // loads are unconditional (of the last tile again behind the end, and of page 0 for a
    // page outside the pool, whose tokens are masked): the next tile's are in flight
    // while one is computed
    Ti tile;
    auto fetch = [&](int n) {
      const int p = __builtin_amdgcn_readlane(page, n), in = __builtin_amdgcn_readlane(inside, n);
      const int64_t at = ((int64_t)(p < 0 || p >= c.num_pages ? 0 : p) * c.page_stride + (int64_t)in * 16 * c.token_stride) * ES;
      load_tile<DIM, FP8>(tile, kc + at, vc + at, offset, step);
    };
    fetch(0);
    for (int n = 0; n < count; ++n) {
      const int p = __builtin_amdgcn_readlane(page, n);
      const int start = (tile0 + (n0 + n) * kWaves) * 16;
      put_tile<DIM, FP8>(tile, corner);
      wave_lds_fence();
      if (n + 1 < count) fetch(n + 1);
      take_tile<DIM, FP8>(corner, q, factor, begin - start, p < 0 || p >= c.num_pages ? 0 : len - start, run, o);
      wave_lds_fence();
    }
  }
  run.l += __shfl_xor(run.l, 16);
  run.l += __shfl_xor(run.l, 32);

  // the waves' results, joined in LDS
  __shared__ float ms[kWaves][16], ls[kWaves][16];
  float* os = reinterpret_cast<float*>(dynamic_lds);  // [wave][heads][PAD], over the waves' corners
  __syncthreads();
  if (r < heads) {
    if (g == 0) ms[wave][r] = run.m, ls[wave][r] = run.l;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < DIM / 16; i += 4) {
        const float4_t w = {o[i][j], o[i + 1][j], o[i + 2][j], o[i + 3][j]};
        *reinterpret_cast<float4_t*>(os + (wave * heads + r) * PAD + out_element<DIM, FP8>(g * 4 + j, i)) = w;
      }
  }
  __syncthreads();
  const float vg = FP8 ? *c.v_amax / 448.0f : 1.0f;
  float* parts = static_cast<float*>(a.workspace);
  float2* heads_ml = reinterpret_cast<float2*>(parts + part_row(a, (int)a.B, 0, splits, 0) * DIM);
  for (int e = threadIdx.x * 4; e < heads * DIM; e += kWaves * 64 * 4) {
    const int h = e / DIM, d = e % DIM;
    float top = kNone, sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ms[w][h]);
    float4_t x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ms[w][h] - top);
      sum += ls[w][h] * f;
      x += *reinterpret_cast<const float4_t*>(os + (w * heads + h) * PAD + d) * f;
    }
    if (only) {
      const float by = sum == 0 ? 0.0f : vg / sum;
      store_out(a.out + (int64_t)b * a.ldo + (int64_t)(head0 + h) * DIM + d, x * by);
      if (a.lse && d == 0)
        a.lse[(int64_t)b * a.q_heads + head0 + h] = sum == 0 ? -INFINITY : top * kLn2 + logf(sum);
    } else {
      const int64_t at = part_row(a, b, head0 + h, splits, split);
      *reinterpret_cast<float4_t*>(parts + at * DIM + d) = x;
      if (d == 0) heads_ml[at] = make_float2(top, sum);
    }
  }
}

// Joins the splits of one query head: each counts 2^(its m - the largest m).  Groups of
// DIM / 4 threads take the splits in turn, then one group their sums.
template <int DIM, bool FP8, int kGroups>
__global__ __launch_bounds__(DIM / 4 * kGroups) void attn_join_kernel(AttnArgs a, Plan plan) {
  constexpr int kLanes = DIM / 4;
  const int splits = plan.splits;
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int start = a.window > 0 ? max(0, len - a.window) / 16 * 16 : 0;
  const int split_tokens = plan.tokens_of(len, a.window), used = (len - start + split_tokens - 1) / split_tokens;
  if (used <= 1) return;
  const float* parts = static_cast<const float*>(a.workspace);
  const float2* ml = reinterpret_cast<const float2*>(parts + part_row(a, (int)gridDim.y, 0, splits, 0) * DIM) +
                     part_row(a, b, h, splits, 0);
  const float* row = parts + part_row(a, b, h, splits, 0) * DIM + d * 4;
  float m = kNone, sum = 0;
  float4_t x = {0, 0, 0, 0};
  for (int s = grp; s < used; s += kGroups) {
    const float2 w = ml[s];
    const float4_t v = *reinterpret_cast<const float4_t*>(row + (int64_t)s * DIM);
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
  const float by = sum == 0 ? 0.0f : (FP8 ? *a.cache.v_amax / 448.0f : 1.0f) / sum;
  store_out(a.out + (int64_t)b * a.ldo + (int64_t)h * DIM + d * 4, x * by);
  if (a.lse && d == 0) a.lse[(int64_t)b * a.q_heads + h] = sum == 0 ? -INFINITY : top * kLn2 + logf(sum);
}

size_t attn_decode_workspace(int64_t B, int q_heads, int kv_heads, int head_dim, int64_t max_len, int64_t window) {
  const int splits = attn_plan(B, q_heads, kv_heads, max_len, window).splits;
  return splits > 1 ? (size_t)B * q_heads * splits * (head_dim + 2) * sizeof(float) : 0;
}

template <int DIM, bool FP8, int kWaves>
static hipError_t launch_waves(const AttnArgs& a, const Plan& plan, hipStream_t stream) {
  const int group = a.q_heads / a.cache.kv_heads;
  const dim3 grid((unsigned)(a.cache.kv_heads * ((group + 15) / 16) * ((a.B * plan.splits + 7) / 8 * 8)));
  auto bytes = [](int heads) {
    return std::max<size_t>((size_t)kWaves * heads * (DIM + 4) * sizeof(float), (size_t)kWaves * Tile<DIM, FP8>::kLdsBytes);
  };
  const size_t lds = bytes(std::min(group, 16));
  hipError_t e = hipSuccess;
  // Above the default bound of dynamic LDS (many heads of 128 or 256).  The bound is the
  // kernel's, for all threads of the process: always that of 16 heads, so that no other call
  // can set it lower between here and the launch.
  if (lds > 48 * 1024)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&attn_decode_kernel<DIM, FP8, kWaves>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(16));
  if (e != hipSuccess) return e;
  attn_decode_kernel<DIM, FP8, kWaves><<<grid, kWaves * 64, lds, stream>>>(a, plan);
  return hipGetLastError();
}

template <int DIM, bool FP8>
static hipError_t launch_dim(const AttnArgs& a, hipStream_t stream) {
  const Plan plan = attn_plan(a.B, a.q_heads, a.cache.kv_heads, a.max_len, a.window);
  // few short sequences: eight waves to a workgroup, so that each has fewer tiles to go through
  const bool few = plan.splits == 1 && a.B * a.q_heads <= 2 * kCUs;
  hipError_t e = few ? launch_waves<DIM, FP8, 8>(a, plan, stream) : launch_waves<DIM, FP8, 4>(a, plan, stream);
  if (e != hipSuccess || plan.splits == 1) return e;
  const dim3 rows(a.q_heads, (unsigned)a.B);
  if (plan.splits <= 16)
    attn_join_kernel<DIM, FP8, 4><<<rows, DIM, 0, stream>>>(a, plan);
  else
    attn_join_kernel<DIM, FP8, 16><<<rows, DIM * 4, 0, stream>>>(a, plan);
  return hipGetLastError();
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream) {
  const bool fp8 = a.cache.dtype == NVFP4_E4M3;
  switch (a.cache.head_dim) {
    case 64: return fp8 ? launch_dim<64, true>(a, stream) : launch_dim<64, false>(a, stream);
    case 128: return fp8 ? launch_dim<128, true>(a, stream) : launch_dim<128, false>(a, stream);
    default: return fp8 ? launch_dim<256, true>(a, stream) : launch_dim<256, false>(a, stream);
  }
}

}  // namespace nvfp4

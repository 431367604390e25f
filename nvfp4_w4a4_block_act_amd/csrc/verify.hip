// Verification of drafted tokens against the target model's logits.
//
// Everything that decides is binary64: a token is the first whose running sum of weights
// passes u times their total, and over a vocabulary of 10^5 the borders lie so close that
// binary32 sums, or exponentials of binary32, would draw another token once in some
// thousand draws.  e^((l - m) / T) is 2^(n + i / 256 + f): the power of i / 256 from a table in
// LDS, 2^f the first four terms of its series (|f| <= 1/512: the rest is below 2^-42 of it).
// (Without a table twelve terms are needed: 186 us against 136 for the sizes below.)
//
// verify_rows: one pass over the logits, and the only one.  A workgroup takes one chunk of
// 8192 logits of one node, 32 to a thread, all loads in flight at once: their maximum, where
// it is, and the sum of exponentials under it.  Where drafts are picked without chance the
// sum leaves out the tokens of the node's own children: these are added one by one in the
// walk, and the last token is drawn from the others, whose sums then need no differences.
// verify_draw: one workgroup a sequence joins its nodes' chunks, walks down the tree (each
// lane of a wave a node), and draws the last token: a running sum over the last node's
// chunks, then over the 8192 logits of one chunk, which is all that is read again.
// With draft logits (chains) the weights after a rejection are max(p - q, 0), which no
// chunk sum of p and q gives: several workgroups of a sequence walk for themselves and sum them, and
// the one that finishes last (a count that verify_rows clears) draws from these sums.
//
// Every sum has a fixed order: results do not depend on timing.
//
// verify_rows is bound by the vector units, and by memory little behind them: 64 x 24 rows of 131072 logits
// (740 MB without those of padded nodes) take 140 us, 5.3 TB/s, with 84 % of the vector units' time in use; 2 x 174
// rows of 100003 (128 MB without draft rows that no child follows) 31.
// verify_draw is bound by its chain of loads, sums and exchanges: 8.3 us for one sequence, 13.3 for 64,
// and 23.0 for 29 of which each sums the residuals of 100003 logits.
#include <algorithm>

#include "common.hpp"
#include "drafts.hpp"
#include "mixers_device.hpp"

namespace nvfp4 {

constexpr int kThreads = 256, kEach = 32, kChunk = kThreads * kEach;
typedef float row4_t __attribute__((ext_vector_type(4), aligned(4)));  // rows begin at any element
constexpr double kLog2eD = 1.4426950408889634074;

struct Part {
  float m;     // largest logit of a chunk
  int32_t at;  // the first that is as large; -1: none is above -inf
  double sum;  // of 2^((l - m) heat)
};

// Numbers of a launch: parts of target rows, parts of draft rows, sums of the rest and how many
// of a sequence's workgroups have theirs.
struct Sizes {
  int chunks, groups;
  Part* p;
  Part* q;
  double* rest;
  uint32_t* done;
};
static int64_t chunks_of(int64_t vocab) { return (vocab + kChunk - 1) / kChunk; }

// 2^(i / kSteps), from the series of the exponential at compile time.
constexpr int kSteps = 256;
struct Powers {
  double at[kSteps];
};
constexpr Powers powers() {
  Powers t{};
  for (int i = 0; i < kSteps; ++i) {
    const double x = i * (0.69314718055994530942 / kSteps);
    double p = 1.0;
    for (int k = 20; k > 0; --k) p = p * x / k + 1.0;
    t.at[i] = p;
  }
  return t;
}
__device__ const Powers kPowers = powers();

// Into LDS, by the whole workgroup; a barrier has to follow.
__device__ __forceinline__ void copy_powers(double* table) {
  for (int i = threadIdx.x; i < kSteps; i += blockDim.x) table[i] = kPowers.at[i];
}

// 2^t for t <= 0, as 2^-1000 below that (and for NaN): t = n + i / kSteps + f, its whole steps from
// the low bits of a sum that leaves no bits behind them.
__device__ __forceinline__ double exp2_below(double t, const double* table) {
  constexpr double kShift = 0x1.8p52 / kSteps, kLn2 = 0.69314718055994530942;
  t = fmax(t, -1000.0);
  const double up = t + kShift;
  const int whole = __double2loint(up);
  const double f = t - (up - kShift);
  const double p = fma(fma(kLn2 * kLn2 * kLn2 / 6, f, kLn2 * kLn2 / 2), f, kLn2);
  const double base = table[whole & (kSteps - 1)];
  const double r = fma(p * f, base, base);
  return __hiloint2double(__double2hiint(r) + (whole & ~(kSteps - 1)) * ((1 << 20) / kSteps), __double2loint(r));
}

// The weight of logit l where the largest is m.  The difference comes first, whose product is never above 0: with
// l heat - m heat in one rounding each the error was that of m heat, which is above every weight's exponent where
// the temperature is below 2^-60 of the logits.  (One instruction less: 149 us against 155 for 64 x 24 x 131072.)
struct Scale {
  double heat, m;
  const double* table;
  __device__ __forceinline__ double of(float l) const { return exp2_below(((double)l - m) * heat, table); }
};
__device__ __forceinline__ Scale scale_of(double heat, float m, const double* table) { return {heat, (double)m, table}; }

// A weight below kLeast is none, and so is a chunk's sum below kLeastSum (one above it has a weight above kLeast): of
// -inf exp2_below leaves 2^-1000, of a chunk in which only turned-down tokens have a logit 2^-987, and a number of 0
// must find neither.
constexpr double kLeastSum = 0x1p-900, kLeast = kLeastSum / (2 * kChunk);
__device__ __forceinline__ double weight_or_none(double w) { return w > kLeast ? w : 0.0; }

// log2(e) / temperature; 0: greedy
__device__ __forceinline__ double heat_of(const VerifyArgs& a, int b) {
  const float t = a.temperature ? a.temperature[b] : 0.0f;
  return t > 0.0f ? kLog2eD / (double)t : 0.0;
}
__device__ __forceinline__ bool greedy(const VerifyArgs& a, int b) { return !(a.temperature && a.temperature[b] > 0.0f); }

__device__ __forceinline__ int parent_of(const VerifyArgs& a, int b, int node) {
  return a.parents ? a.parents[(int64_t)b * a.nodes + node] : node - 1;
}

// A lane's node: its parent, -1 for node 0 of a sequence, -2 for what is no node.
__device__ __forceinline__ int lane_parent(const VerifyArgs& a, int b, int lane) {
  if (lane >= a.nodes) return -2;
  const int p = parent_of(a, b, lane);
  return lane == 0 ? (p == -1 ? -1 : -2) : (p >= 0 && p < lane ? p : -2);
}
__device__ __forceinline__ int64_t lane_token(const VerifyArgs& a, int b, int lane, int parent) {
  const int64_t t = parent >= 0 ? a.drafts[(int64_t)b * a.nodes + lane] : -1;
  return t >= 0 && t < a.vocab ? t : -1;
}

// Four logits of a row of `count` from `at` on, -inf behind its end.
__device__ __forceinline__ row4_t load4(const float* from, int at, int count) {
  if (at + 4 <= count) return *reinterpret_cast<const row4_t*>(from + at);
  row4_t w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = at + j < count ? from[at + j] : -INFINITY;
  return w;
}

// Sum over the workgroup's threads, in all of them.
__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(kThreads) void verify_rows_kernel(VerifyArgs a, Sizes z) {
  const int chunk = blockIdx.x % z.chunks;
  int row = blockIdx.x / z.chunks;
  const int rows = a.B * a.nodes;
  const bool is_draft = row >= rows;
  row -= is_draft ? rows : 0;
  const int b = row / a.nodes, node = row % a.nodes;
  const int lane = threadIdx.x % 64;
  const int64_t first = (int64_t)chunk * kChunk;
  const float* from = (is_draft ? a.draft + row * a.ldd : a.logits + row * a.ld) + first;
  const int count = (int)min((int64_t)kChunk, a.vocab - first);
  float x[kEach];
  auto load = [&] {
#pragma unroll
    for (int k = 0; k < kEach / 4; ++k) {
      const row4_t w = load4(from, (k * kThreads + threadIdx.x) * 4, count);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * k + j] = w[j];
    }
  };
  // Where the launch does not fill the GPU the logits are on their way before it is known
  // whether anybody asks for them: 14.2 us in all for 1 x 8 x 32000, otherwise 14.5, 14.8 and 15.0 for
  // 2 x 8 x 100003; 18.9 and 18.7 for 8 x 8 x 100003, with 832 workgroups.
  const bool early = gridDim.x <= kCUs;
  if (early) load();
  if (a.draft && chunk == 0 && node == 0 && !is_draft && threadIdx.x == 0) z.done[b] = 0;
  const int parent = lane_parent(a, b, lane);
  const int64_t token = lane_token(a, b, lane, parent);
  uint64_t kids = __ballot(parent == node && token >= 0);
  const bool is_greedy = greedy(a, b);
  if (!early) {
    if (__shfl(parent, node) == -2 || (is_draft && (is_greedy || kids == 0))) return;
    load();
  }
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < kEach; ++e) m = fmaxf(m, x[e]);
  const float mine = m;
  __shared__ float ms[kThreads / 64];
  __shared__ int found;  // where the largest is
  __shared__ double table[kSteps];
  copy_powers(table);
#pragma unroll
  for (int s = 1; s < 64; s *= 2) m = fmaxf(m, __shfl_xor(m, s));
  if (lane == 0) ms[threadIdx.x / 64] = m;
  if (threadIdx.x == 0) found = 0x7FFFFFFF;
  __syncthreads();
  m = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
  if (mine == m && m > -INFINITY) {
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int e = kEach - 1; e >= 0; --e)
      if (x[e] == m) at = (e / 4 * kThreads + threadIdx.x) * 4 + e % 4;
    atomicMin(&found, at);
  }

  double sum = 0;
  if (!is_greedy) {
    if (!a.draft) {
      for (; kids; kids &= kids - 1) {
        const int64_t t = __shfl(token, __builtin_ctzll(kids)) - first;
        if (t < 0 || t >= count || (t / 4) % kThreads != threadIdx.x) continue;
        const int mine = (int)(t / 4 / kThreads * 4 + t % 4);
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          if (e == mine) x[e] = -INFINITY;
      }
    }
    const Scale scale = scale_of(heat_of(a, b), m > -INFINITY ? m : 0.0f, table);
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum += scale.of(x[e]);
    __shared__ double sums[kThreads / 64];
    sum = block_sum(sum, sums);
  } else {
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const Part part = {m, m > -INFINITY ? (int32_t)(found + first) : -1, sum};
    (is_draft ? z.q : z.p)[(int64_t)row * z.chunks + chunk] = part;
  }
}

// The draw's kernel takes one chunk with many threads, so that each has only a few of its logits: its code
// is run through once, by few workgroups, and fetching it sets their time (39 KB of code, with 256 threads,
// took 13 and 21 us for one and 64 sequences, 10 KB 9 and 14).
template <bool DRAWN>
struct Draw {
  static constexpr int kThreads = 1024, kEach = kChunk / kThreads, kWaves = kThreads / 64, kRuns = kEach / 4;
  static constexpr int kSub = kThreads / NVFP4_MAX_NODES;  // threads that join a node's chunks
};

// What a walk ends with, in LDS.
struct Walk {
  double table[kSteps];
  float m[2][NVFP4_MAX_NODES];     // largest logit of each node's row; [1]: of its draft row
  double sum[2][NVFP4_MAX_NODES];  // of the row's weights, as verify_rows left them
  int at[NVFP4_MAX_NODES];         // where the largest logit is
  int tried[NVFP4_MAX_NODES];      // tokens of the last node's children
  int tries, node, count;          // count 0: a padded sequence
};

// The walk of sequence b by a workgroup; `store`: writes the outputs it decides.  Every number
// a step may need is on its way before the first: each lane has its own node's, as a child.
template <bool DRAWN>
__device__ __forceinline__ void walk_tree(const VerifyArgs& a, const Sizes& z, int b, bool store, Walk& w) {
  constexpr int kSub = Draw<DRAWN>::kSub;
  const int lane = threadIdx.x % 64, row = threadIdx.x / kSub, sub = threadIdx.x % kSub;
  const Part none = {-INFINITY, -1, 0.0};
  const int64_t at_parts = ((int64_t)b * a.nodes + row) * z.chunks;
  // the first chunk of each thread (a row that nobody asked for holds anything)
  const bool one = row < a.nodes && sub < z.chunks;
  Part ahead[2] = {one ? z.p[at_parts + sub] : none, none};
  if (DRAWN && one) ahead[1] = z.q[at_parts + sub];
  const float number = a.temperature && lane < a.nodes ? a.uniforms[(int64_t)b * (a.nodes + 1) + lane] : 0.0f;
  const int parent = lane_parent(a, b, lane);
  const int token = (int)lane_token(a, b, lane, parent);
  const bool is_greedy = greedy(a, b);
  const double heat = heat_of(a, b);
  float l[2] = {-INFINITY, -INFINITY};
  if (!is_greedy && token >= 0) {
    const int64_t up = (int64_t)b * a.nodes + parent;
    l[0] = a.logits[up * a.ld + token];
    if (DRAWN) l[1] = a.draft[up * a.ldd + token];
  }
  copy_powers(w.table);
  uint64_t asked = __ballot(parent != -2);
  if (threadIdx.x < NVFP4_MAX_NODES) w.m[0][lane] = w.m[1][lane] = -INFINITY, w.sum[0][lane] = w.sum[1][lane] = 0.0;
  __syncthreads();
#pragma unroll 1
  for (int d = 0; d < (DRAWN ? 2 : 1); ++d) {
    if (d == 1) {
      uint64_t inner = 0;  // of draft rows only those of nodes that have children
#pragma unroll 1
      for (int i = 0; i < a.nodes; ++i) inner |= __ballot(parent == i && token >= 0) ? 1ull << i : 0;
      asked &= inner;
    }
    if (row < a.nodes && (asked >> row & 1)) {
      const Part* parts = (d ? z.q : z.p) + at_parts;
      const Part first = d ? ahead[1] : ahead[0];
      float m = first.m;
      int at = first.at;
#pragma unroll 1
      for (int c = sub + kSub; c < z.chunks; c += kSub)
        if (parts[c].m > m) m = parts[c].m, at = parts[c].at;
#pragma unroll
      for (int s = 1; s < kSub; s *= 2) {
        const float om = __shfl_xor(m, s);
        const int oat = __shfl_xor(at, s);
        if (om > m || (om == m && (uint32_t)oat < (uint32_t)at)) m = om, at = oat;
      }
      double sum = 0;
      if (m > -INFINITY && !is_greedy) {
        const Scale under = scale_of(heat, m, w.table);
        Part p = first;
#pragma unroll 1
        for (int c = sub;;) {
          if (p.m > -INFINITY) sum += p.sum * under.of(p.m);
          c += kSub;
          if (c >= z.chunks) break;
          p = parts[c];
        }
      }
#pragma unroll
      for (int s = 1; s < kSub; s *= 2) sum += __shfl_xor(sum, s);
      if (sub == 0) {
        w.m[d][row] = m, w.sum[d][row] = sum;
        if (d == 0) w.at[row] = at;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    // the lane's node, as a child: its weights under its parent
    double mine[2] = {0, 0};
#pragma unroll
    for (int d = 0; d < (DRAWN ? 2 : 1); ++d)
      if (l[d] > -INFINITY) mine[d] = weight_or_none(scale_of(heat, w.m[d][parent], w.table).of(l[d]));
    bool again = false;  // an earlier child of the same parent has the same token
    if (!DRAWN)
#pragma unroll 4
      for (int i = 1; i < a.nodes; ++i) {
        const int t = __builtin_amdgcn_readlane(token, i), up = __builtin_amdgcn_readlane(parent, i);
        again |= i < lane && t >= 0 && up == parent && t == token;
      }
    int node = 0, count = __shfl(parent, 0) == -1 ? 1 : 0;
    uint64_t kids = 0;
    for (int left = a.nodes; count > 0 && left > 0; --left) {
      kids = __ballot(parent == node && token >= 0 && !again);
      int taken = -1;
      if (is_greedy) {
        const uint64_t best = __ballot(parent == node && token >= 0 && token == w.at[node]);
        if (best) taken = __builtin_ctzll(best);
      } else if (kids) {
        const double u = fmin(fmax((double)__shfl(number, node), 0.0), 1.0 - 0x1p-24);
        if (DRAWN) {
          const int kid = __builtin_ctzll(kids);
          const double pk = __shfl(mine[0], kid) * w.sum[1][node], qk = __shfl(mine[1], kid) * w.sum[0][node];
          if (u * qk < pk) taken = kid;
          kids = 1ull << kid;
        } else {
          double total = w.sum[0][node], mass = 0;
          for (uint64_t k = kids; k; k &= k - 1) total += __shfl(mine[0], __builtin_ctzll(k));
          for (uint64_t k = kids; k && taken < 0; k &= k - 1) {
            const int kid = __builtin_ctzll(k);
            mass += __shfl(mine[0], kid);
            if (u * total < mass) taken = kid;
          }
        }
      }
      if (taken < 0) break;
      node = taken;
      const int t = __shfl(token, taken);
      if (store && lane == 0) {
        a.tokens[(int64_t)b * a.nodes + count - 1] = t;
        a.path[(int64_t)b * a.nodes + count] = taken;
      }
      ++count;
    }
    if (kids >> lane & 1) w.tried[__popcll(kids & ((1ull << lane) - 1))] = token;
    if (lane == 0) w.node = node, w.count = count, w.tries = is_greedy ? 0 : __popcll(kids);
    if (store) {
      const int64_t at = (int64_t)b * a.nodes;
      if (lane == 0) a.counts[b] = count;
      if (lane == 0 && count > 0) a.path[at] = 0;
      if (lane >= count && lane < a.nodes) a.path[at + lane] = -1, a.tokens[at + lane] = -1;
    }
  }
  __syncthreads();
}

// The weights after the last node: of p, or max(p - q, 0).
struct Last {
  const float* l;
  const float* l2;  // null: no residual
  Scale p, q;
  double per, per2;  // 1 / sums
};
template <bool DRAWN>
__device__ __forceinline__ Last last_of(const VerifyArgs& a, const Walk& w, int b) {
  const int64_t row = (int64_t)b * a.nodes + w.node;
  const bool rest = DRAWN && w.tries > 0;
  const double heat = heat_of(a, b);
  return {a.logits + row * a.ld,
          rest ? a.draft + row * a.ldd : nullptr,
          scale_of(heat, w.m[0][w.node], w.table),
          scale_of(heat, rest ? w.m[1][w.node] : 0.0f, w.table),
          rest ? 1.0 / w.sum[0][w.node] : 1.0,
          rest && w.sum[1][w.node] > 0.0 ? 1.0 / w.sum[1][w.node] : 0.0};
}

// Weights of the chunk that begins at column `first`, this thread's runs of four.
template <bool DRAWN>
struct Weights {
  double w[Draw<DRAWN>::kEach];
};
template <bool DRAWN>
__device__ __forceinline__ void weights_of(const VerifyArgs& a, const Last& last, int64_t first, Weights<DRAWN>& r) {
  const int count = (int)min((int64_t)kChunk, a.vocab - first);
  row4_t x[Draw<DRAWN>::kRuns], y[Draw<DRAWN>::kRuns];
#pragma unroll
  for (int k = 0; k < Draw<DRAWN>::kRuns; ++k) {
    x[k] = load4(last.l + first, (k * Draw<DRAWN>::kThreads + threadIdx.x) * 4, count);
    y[k] = DRAWN && last.l2 ? load4(last.l2 + first, (k * Draw<DRAWN>::kThreads + threadIdx.x) * 4, count) : x[k];
  }
#pragma unroll
  for (int e = 0; e < Draw<DRAWN>::kEach; ++e) r.w[e] = weight_or_none(last.p.of(x[e / 4][e % 4]));
  if (DRAWN && last.l2) {
#pragma unroll
    for (int e = 0; e < Draw<DRAWN>::kEach; ++e) {
      const float l = y[e / 4][e % 4];
      r.w[e] = fmax(r.w[e] * last.per - weight_or_none(last.q.of(l)) * last.per2, 0.0);
    }
  }
}

// The sum over the lanes before this one.
__device__ __forceinline__ double sum_before(double x, int lane) {
  double run = x;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const double y = __shfl_up(run, s);
    if (lane >= s) run += y;
  }
  return run - x;
}

// One workgroup a sequence, or with draft logits several, which share its chunks.
template <bool DRAWN>
__global__ __launch_bounds__(Draw<DRAWN>::kThreads) void verify_draw_kernel(VerifyArgs a, Sizes z) {
  const int b = DRAWN ? blockIdx.x / z.groups : blockIdx.x, own = DRAWN ? blockIdx.x % z.groups : 0;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  __shared__ Walk w;
  __shared__ double sums[Draw<DRAWN>::kRuns][Draw<DRAWN>::kWaves];
  __shared__ bool is_last;
  if (DRAWN && own > 0 && greedy(a, b)) return;
  walk_tree<DRAWN>(a, z, b, own == 0, w);
  if (w.count == 0 || (DRAWN && own > 0 && w.tries == 0)) return;
  int64_t* out = a.tokens + (int64_t)b * a.nodes + w.count - 1;
  if (greedy(a, b)) {
    if (threadIdx.x == 0) *out = w.at[w.node];
    return;
  }
  const Last last = last_of<DRAWN>(a, w, b);
  const Part* parts = z.p + ((int64_t)b * a.nodes + w.node) * z.chunks;
  const double* rests = z.rest + (int64_t)b * z.chunks;
  const double u = fmin(fmax((double)a.uniforms[(int64_t)b * (a.nodes + 1) + a.nodes], 0.0), 1.0 - 0x1p-24);
  Weights<DRAWN> r;
  double four[Draw<DRAWN>::kRuns];
  auto add_up = [&] {  // the sums of the runs, of each wave
#pragma unroll
    for (int k = 0; k < Draw<DRAWN>::kRuns; ++k) {
      double s = four[k] = (r.w[4 * k] + r.w[4 * k + 1]) + (r.w[4 * k + 2] + r.w[4 * k + 3]);
#pragma unroll
      for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m);
      if (lane == 0) sums[k][wave] = s;
    }
    __syncthreads();
  };
  int chunk = own;
  double left = 0;
  // With draft logits and a rejection the workgroup's turns sum its own chunks, and the workgroup that finishes
  // last takes one more, in which it draws; otherwise there is only that one.
  bool draw = !(DRAWN && last.l2);
#pragma unroll 1
  for (;;) {
    if (draw) {
      // The chunk, found by every wave alike: a run of chunks to each lane.
      const int each = (z.chunks + 63) / 64, c0 = lane * each, c1 = min(c0 + each, z.chunks);
      auto chunk_sum = [&](int c) {
        if (DRAWN && last.l2) return __hip_atomic_load(&rests[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const double s = parts[c].m > -INFINITY ? parts[c].sum * last.p.of(parts[c].m) : 0.0;
        return s > kLeastSum ? s : 0.0;
      };
      double sum = 0;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) sum += chunk_sum(c);
      const double before = sum_before(sum, lane), target = u * __shfl(before + sum, 63);
      const uint64_t some = __ballot(sum > 0.0), above = __ballot(sum > 0.0 && before + sum > target);
      if (some == 0) {  // no weight anywhere: the largest logit
        if (threadIdx.x == 0) *out = w.at[w.node];
        return;
      }
      // (none above only by rounding: then the last one with a weight)
      const int owner = above ? __builtin_ctzll(above) : 63 - __builtin_clzll(some);
      chunk = c0, left = target - before;
#pragma unroll 1
      for (int c = c0; c < c1 && each > 1; ++c) {
        const double s = chunk_sum(c);
        if (s <= 0.0) continue;
        chunk = c;
        if (s > left) break;
        if (c + 1 < c1) left -= s;
      }
      chunk = __shfl(chunk, owner);
      left = __shfl(left, owner);
    }
    const int64_t first = (int64_t)chunk * kChunk;
    weights_of<DRAWN>(a, last, first, r);
    if (!DRAWN) {
#pragma unroll 1
      for (int i = 0; i < w.tries; ++i) {
        const int64_t t = w.tried[i] - first;
        if (t < 0 || t >= kChunk || (t / 4) % Draw<DRAWN>::kThreads != threadIdx.x) continue;
        const int mine = (int)(t / 4 / Draw<DRAWN>::kThreads * 4 + t % 4);
#pragma unroll
        for (int e = 0; e < Draw<DRAWN>::kEach; ++e)
          if (e == mine) r.w[e] = 0.0;
      }
    }
    add_up();
    if (draw) break;
    chunk += z.groups;
    const bool more = chunk < z.chunks;
    if (threadIdx.x == 0) {
      double sum = 0;
      for (int i = 0; i < Draw<DRAWN>::kRuns * Draw<DRAWN>::kWaves; ++i) sum += sums[i / Draw<DRAWN>::kWaves][i % Draw<DRAWN>::kWaves];
      // Each workgroup's sums come before its count, and all counts before the last one reads the sums.  (One thread's
      // release and acquire: 54.4 us, as with the order left to the instructions' own waits.)
      __hip_atomic_store(&z.rest[(int64_t)b * z.chunks + chunk - z.groups], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (!more)
        is_last = __hip_atomic_fetch_add(&z.done[b], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 == (uint32_t)z.groups;
    }
    __syncthreads();
    if (more) continue;
    if (!is_last) return;
    draw = true;
  }

  // The token in the chunk: runs of 4096 logits, a wave's part of a run, lanes, fours.  Every wave finds the
  // part alike, a lane to each.
  static_assert(Draw<DRAWN>::kRuns * Draw<DRAWN>::kWaves <= 64, "a lane to each part");
  const double part_sum = lane < Draw<DRAWN>::kRuns * Draw<DRAWN>::kWaves ? sums[lane / Draw<DRAWN>::kWaves][lane % Draw<DRAWN>::kWaves] : 0.0;
  const double part_before = sum_before(part_sum, lane);
  const uint64_t filled = __ballot(part_sum > 0.0), past = __ballot(part_sum > 0.0 && part_before + part_sum > left);
  if (filled == 0) {
    if (threadIdx.x == 0) *out = w.at[w.node];
    return;
  }
  const int part = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(filled);
  const double in = left - __shfl(part_before, part);
  if (wave != part % Draw<DRAWN>::kWaves) return;
  double mine[4] = {0, 0, 0, 0}, total = 0;
#pragma unroll
  for (int k = 0; k < Draw<DRAWN>::kRuns; ++k)
    if (k == part / Draw<DRAWN>::kWaves) {
      total = four[k];
#pragma unroll
      for (int j = 0; j < 4; ++j) mine[j] = r.w[4 * k + j];
    }
  const double before = sum_before(total, lane);
  const uint64_t any = __ballot(total > 0.0), over = __ballot(total > 0.0 && before + total > in);
  if (lane != (over ? __builtin_ctzll(over) : 63 - __builtin_clzll(any))) return;
  int best = 0;
  double rest = in - before;
  bool found = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!found && mine[j] > 0.0) best = j, found = mine[j] > rest;
    rest -= mine[j];
  }
  *out = (int64_t)chunk * kChunk + ((part / Draw<DRAWN>::kWaves) * Draw<DRAWN>::kThreads + wave * 64 + lane) * 4 + best;
}

size_t verify_workspace(int64_t B, int nodes, int64_t vocab, bool sampled) {
  const size_t chunks = (size_t)chunks_of(vocab), rows = (size_t)B * nodes, parts = rows * chunks * sizeof(Part);
  return sampled ? 2 * parts + ((size_t)B * (chunks * sizeof(double) + sizeof(uint32_t)) + 15) / 16 * 16 : parts;
}

int64_t verify_groups(int64_t B, int nodes, int64_t vocab, bool sampled) {
  return B * nodes * (sampled ? 2 : 1) * chunks_of(vocab);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  const int rows = a.B * a.nodes, chunks = (int)chunks_of(a.vocab);
  Part* p = static_cast<Part*>(a.workspace);
  Part* q = a.draft ? p + (int64_t)rows * chunks : nullptr;
  double* rest = a.draft ? reinterpret_cast<double*>(q + (int64_t)rows * chunks) : nullptr;
  // as many workgroups for a sequence as the GPU runs at once, one on a CU
  const int groups = std::min(chunks, std::max(1, kCUs / a.B));
  const Sizes z = {chunks, groups, p, q, rest, a.draft ? reinterpret_cast<uint32_t*>(rest + (int64_t)a.B * chunks) : nullptr};
  verify_rows_kernel<<<dim3((unsigned)((int64_t)rows * (a.draft ? 2 : 1) * chunks)), kThreads, 0, stream>>>(a, z);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.draft)
    verify_draw_kernel<true><<<dim3((unsigned)((int64_t)a.B * groups)), Draw<true>::kThreads, 0, stream>>>(a, z);
  else
    verify_draw_kernel<false><<<dim3((unsigned)a.B), Draw<false>::kThreads, 0, stream>>>(a, z);
  return hipGetLastError();
}

}  // namespace nvfp4

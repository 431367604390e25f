// Verification of drafted tokens against the target model's logits.
//
// Everything that decides is binary64: a token is the first whose running sum of weights
// passes u times their total, and over a vocabulary of 10^5 the borders lie so close that
// binary32 sums, or exponentials of binary32, would draw another token once in some
// thousand draws.  e^((l - m) / T) is 2^(n + f), 2^f the first twelve terms of its power
// series (|f| <= 1/2: the rest is below 2^-47 of it).
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
// chunk sum of p and q gives: verify_rest sums them chunk by chunk, after a walk of its own
// in each workgroup, and verify_draw takes these sums.
//
// Every sum has a fixed order: results do not depend on timing.
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

// Numbers of a launch: parts of target rows, parts of draft rows, sums of the rest.
struct Sizes {
  int chunks;
  Part* p;
  Part* q;
  double* rest;
};
static int64_t chunks_of(int64_t vocab) { return (vocab + kChunk - 1) / kChunk; }

// 2^t, t <= 0 (NaN counts as 2^-1080: 0)
__device__ __forceinline__ double exp2_below(double t) {
  t = fmax(t, -1080.0);
  const double n = rint(t), x = (t - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = fma(p, x, 1.0 / 3628800.0);
  p = fma(p, x, 1.0 / 362880.0);
  p = fma(p, x, 1.0 / 40320.0);
  p = fma(p, x, 1.0 / 5040.0);
  p = fma(p, x, 1.0 / 720.0);
  p = fma(p, x, 1.0 / 120.0);
  p = fma(p, x, 1.0 / 24.0);
  p = fma(p, x, 1.0 / 6.0);
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  p = fma(p, x, 1.0);
  return ldexp(p, (int)n);
}

__device__ __forceinline__ double weight(float l, float m, double heat) {
  return exp2_below(((double)l - (double)m) * heat);
}

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
  const int parent = lane_parent(a, b, lane);
  const int64_t token = lane_token(a, b, lane, parent);
  uint64_t kids = __ballot(parent == node && token >= 0);
  const bool is_greedy = greedy(a, b);
  if (__shfl(parent, node) == -2) return;
  if (is_draft && (is_greedy || kids == 0)) return;

  const int64_t first = (int64_t)chunk * kChunk;
  const float* from = (is_draft ? a.draft + row * a.ldd : a.logits + row * a.ld) + first;
  const int count = (int)min((int64_t)kChunk, a.vocab - first);
  float x[kEach];
#pragma unroll
  for (int k = 0; k < kEach / 4; ++k) {
    const int at = (k * kThreads + threadIdx.x) * 4;
    if (at + 4 <= count) {
      const row4_t w = *reinterpret_cast<const row4_t*>(from + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * k + j] = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * k + j] = at + j < count ? from[at + j] : -INFINITY;
    }
  }
  float m = -INFINITY;
  int at = -1;
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (x[e] > m) m = x[e], at = (e / 4 * kThreads + threadIdx.x) * 4 + e % 4;
  __shared__ float ms[kThreads / 64];
  __shared__ int ats[kThreads / 64];
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const float om = __shfl_xor(m, s);
    const int oat = __shfl_xor(at, s);
    if (om > m || (om == m && (uint32_t)oat < (uint32_t)at)) m = om, at = oat;
  }
  if (lane == 0) ms[threadIdx.x / 64] = m, ats[threadIdx.x / 64] = at;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w)
    if (ms[w] > m || (ms[w] == m && (uint32_t)ats[w] < (uint32_t)at)) m = ms[w], at = ats[w];

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
    const double heat = heat_of(a, b);
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum += weight(x[e], m, heat);
    __shared__ double sums[kThreads / 64];
    sum = block_sum(sum, sums);
  }
  if (threadIdx.x == 0) {
    const Part part = {m, at < 0 ? -1 : (int32_t)(at + first), sum};
    (is_draft ? z.q : z.p)[(int64_t)row * z.chunks + chunk] = part;
  }
}

// What a walk ends with, in LDS.
struct Walk {
  float m[2][NVFP4_MAX_NODES];     // largest logit of each node's row; [1]: of its draft row
  double sum[2][NVFP4_MAX_NODES];  // of the row's weights, as verify_rows left them
  int at[NVFP4_MAX_NODES];         // where the largest logit is
  int64_t tried[NVFP4_MAX_NODES];  // tokens of the last node's children
  int tries, node, count;          // count 0: a padded sequence
};

// The walk of sequence b by a workgroup; `store`: writes the outputs it decides.
__device__ __forceinline__ void walk_tree(const VerifyArgs& a, const Sizes& z, int b, bool store, Walk& w) {
  // four threads a node: its row's chunks
  const int row = threadIdx.x / 4, sub = threadIdx.x % 4;
  const bool is_greedy = greedy(a, b);
  const double heat = heat_of(a, b);
  const int lane = threadIdx.x % 64;
  const int parent = lane_parent(a, b, lane);
  const int64_t token = lane_token(a, b, lane, parent);
  uint64_t inner = 0;  // nodes that have children
  for (int i = 0; i < a.nodes; ++i) inner |= __ballot(parent == i && token >= 0) ? 1ull << i : 0;
  const uint64_t nodes = __ballot(parent != -2);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    if (d == 1 && (!a.draft || is_greedy)) break;
    const Part* parts = (d ? z.q : z.p) + ((int64_t)b * a.nodes + row) * z.chunks;
    const bool here = row < a.nodes && ((d ? inner & nodes : nodes) >> row & 1);
    float m = -INFINITY;
    int at = -1;
    if (here) {
      for (int c = sub; c < z.chunks; c += 4)
        if (parts[c].m > m) m = parts[c].m, at = parts[c].at;
    }
#pragma unroll
    for (int s = 1; s < 4; s *= 2) {
      const float om = __shfl_xor(m, s);
      const int oat = __shfl_xor(at, s);
      if (om > m || (om == m && (uint32_t)oat < (uint32_t)at)) m = om, at = oat;
    }
    double sum = 0;
    if (here && !is_greedy)
      for (int c = sub; c < z.chunks; c += 4)
        if (parts[c].m > -INFINITY) sum += parts[c].sum * weight(parts[c].m, m, heat);
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (sub == 0) {
      w.m[d][row] = m, w.sum[d][row] = sum;
      if (d == 0) w.at[row] = at;
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    // the lane's node, as a child: its weights under its parent
    double p = 0, q = 0;
    if (token >= 0 && !is_greedy) {
      const int64_t up = (int64_t)b * a.nodes + parent;
      const float l = a.logits[up * a.ld + token];
      p = l > -INFINITY ? weight(l, w.m[0][parent], heat) : 0.0;
      if (a.draft) {
        const float l2 = a.draft[up * a.ldd + token];
        q = l2 > -INFINITY ? weight(l2, w.m[1][parent], heat) : 0.0;
      }
    }
    bool again = false;  // an earlier child of the same parent has the same token
    if (!a.draft)
      for (int i = 1; i < a.nodes; ++i) {
        const int64_t t = __shfl(token, i);
        const int up = __shfl(parent, i);
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
        const double u = fmin(fmax((double)a.uniforms[(int64_t)b * (a.nodes + 1) + node], 0.0), 1.0 - 0x1p-24);
        if (a.draft) {
          const int kid = __builtin_ctzll(kids);
          const double pk = __shfl(p, kid) * w.sum[1][node], qk = __shfl(q, kid) * w.sum[0][node];
          if (u * qk < pk) taken = kid;
          kids = 1ull << kid;
        } else {
          double total = w.sum[0][node], mass = 0;
          for (uint64_t k = kids; k; k &= k - 1) total += __shfl(p, __builtin_ctzll(k));
          for (uint64_t k = kids; k && taken < 0; k &= k - 1) {
            const int kid = __builtin_ctzll(k);
            mass += __shfl(p, kid);
            if (u * total < mass) taken = kid;
          }
        }
      }
      if (taken < 0) break;
      node = taken;
      const int64_t t = __shfl(token, taken);
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

// The weight of token t (a column of the vocabulary) after the last node.
struct Last {
  const float* l;
  const float* l2;  // null: no residual
  float m, m2;
  double heat, sum, sum2;
  __device__ __forceinline__ double of(int64_t t) const {
    const float x = l[t];
    const double p = x > -INFINITY ? weight(x, m, heat) : 0.0;
    if (!l2) return p;
    const float y = l2[t];
    return fmax(p / sum - (y > -INFINITY ? weight(y, m2, heat) / sum2 : 0.0), 0.0);
  }
};
__device__ __forceinline__ Last last_of(const VerifyArgs& a, const Walk& w, int b) {
  const int64_t row = (int64_t)b * a.nodes + w.node;
  const bool rest = a.draft && w.tries > 0;
  return {a.logits + row * a.ld, rest ? a.draft + row * a.ldd : nullptr, w.m[0][w.node], rest ? w.m[1][w.node] : 0.0f,
          heat_of(a, b), w.sum[0][w.node], rest ? w.sum[1][w.node] : 0.0};
}

// Sums of max(p - q, 0) by chunk.
__global__ __launch_bounds__(kThreads) void verify_rest_kernel(VerifyArgs a, Sizes z) {
  const int b = blockIdx.x / z.chunks, chunk = blockIdx.x % z.chunks;
  __shared__ Walk w;
  __shared__ double sums[kThreads / 64];
  if (greedy(a, b)) return;
  walk_tree(a, z, b, false, w);
  if (w.count == 0 || w.tries == 0) return;
  const Last last = last_of(a, w, b);
  const int64_t first = (int64_t)chunk * kChunk;
  const int count = (int)min((int64_t)kChunk, a.vocab - first);
  double sum = 0;
#pragma unroll 4
  for (int k = 0; k < kEach; ++k) {
    const int at = k * kThreads + threadIdx.x;
    if (at < count) sum += last.of(first + at);
  }
  sum = block_sum(sum, sums);
  if (threadIdx.x == 0) z.rest[(int64_t)b * z.chunks + chunk] = sum;
}

// First place whose running sum of the threads' values is above u times their total (or `target`
// if that is not negative): the thread, and what is left of the target at its start.
struct Found {
  int thread;  // -1: all are 0
  double left;
};
__device__ __forceinline__ Found find_thread(double x, double u, double target, double (&scan)[kThreads]) {
  __syncthreads();
  scan[threadIdx.x] = x;
  __syncthreads();
  for (int s = 1; s < kThreads; s *= 2) {
    const double y = threadIdx.x >= s ? scan[threadIdx.x - s] : 0.0;
    __syncthreads();
    scan[threadIdx.x] += y;
    __syncthreads();
  }
  if (target < 0) target = u * scan[kThreads - 1];
  __shared__ Found found;
  __shared__ int last;
  if (threadIdx.x == 0) found = {-1, 0.0}, last = -1;
  __syncthreads();
  const double before = threadIdx.x ? scan[threadIdx.x - 1] : 0.0;
  if (x > 0.0) atomicMax(&last, (int)threadIdx.x);
  if (before <= target && scan[threadIdx.x] > target) found = {(int)threadIdx.x, target - before};
  __syncthreads();
  Found f = found;
  if (f.thread < 0 && last >= 0) f = {last, __builtin_inf()};  // rounding: the last one with a weight
  return f;
}

__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, Sizes z) {
  const int b = blockIdx.x;
  __shared__ Walk w;
  __shared__ double scan[kThreads];
  __shared__ int chosen;
  __shared__ double rest;
  walk_tree(a, z, b, true, w);
  if (w.count == 0) return;
  int64_t* out = a.tokens + (int64_t)b * a.nodes + w.count - 1;
  if (greedy(a, b)) {
    if (threadIdx.x == 0) *out = w.at[w.node];
    return;
  }
  const Last last = last_of(a, w, b);
  const Part* parts = z.p + ((int64_t)b * a.nodes + w.node) * z.chunks;
  const double* rests = z.rest + (int64_t)b * z.chunks;
  const double u = fmin(fmax((double)a.uniforms[(int64_t)b * (a.nodes + 1) + a.nodes], 0.0), 1.0 - 0x1p-24);
  auto chunk_sum = [&](int c) {
    return last.l2 ? rests[c] : (parts[c].m > -INFINITY ? parts[c].sum * weight(parts[c].m, last.m, last.heat) : 0.0);
  };
  // the chunk: a run of chunks to each thread
  const int each = (z.chunks + kThreads - 1) / kThreads, c0 = threadIdx.x * each, c1 = min(c0 + each, z.chunks);
  double sum = 0;
  for (int c = c0; c < c1; ++c) sum += chunk_sum(c);
  Found f = find_thread(sum, u, -1.0, scan);
  if (f.thread < 0) {  // no weight anywhere: the largest logit
    if (threadIdx.x == 0) *out = w.at[w.node];
    return;
  }
  if ((int)threadIdx.x == f.thread) {
    int best = c0;
    double left = f.left;
    for (int c = c0; c < c1; ++c) {
      const double s = chunk_sum(c);
      if (s <= 0.0) continue;
      best = c;
      if (s > left) break;
      left -= s;
    }
    chosen = best, rest = left;
  }
  __syncthreads();
  // the token in it: a run of 32 to each thread
  const int64_t first = (int64_t)chosen * kChunk + threadIdx.x * kEach;
  const int count = (int)max((int64_t)0, min((int64_t)kEach, a.vocab - first));
  const int tries = last.l2 ? 0 : w.tries;
  auto of = [&](int64_t t) {
    for (int i = 0; i < tries; ++i)
      if (w.tried[i] == t) return 0.0;
    return last.of(t);
  };
  sum = 0;
  for (int e = 0; e < count; ++e) sum += of(first + e);
  f = find_thread(sum, 0.0, rest, scan);
  if (f.thread < 0) {
    if (threadIdx.x == 0) *out = w.at[w.node];
    return;
  }
  if ((int)threadIdx.x == f.thread) {
    int64_t best = first;
    double left = f.left;
    for (int e = 0; e < count; ++e) {
      const double s = of(first + e);
      if (s <= 0.0) continue;
      best = first + e;
      if (s > left) break;
      left -= s;
    }
    *out = best;
  }
}

size_t verify_workspace(int64_t B, int nodes, int64_t vocab, bool sampled) {
  const size_t chunks = (size_t)chunks_of(vocab), rows = (size_t)B * nodes;
  return rows * chunks * sizeof(Part) * (sampled ? 2 : 1) + (sampled ? ((size_t)B * chunks * sizeof(double) + 15) / 16 * 16 : 0);
}

int64_t verify_groups(int64_t B, int nodes, int64_t vocab, bool sampled) {
  return B * nodes * (sampled ? 2 : 1) * chunks_of(vocab);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  const int rows = a.B * a.nodes, chunks = (int)chunks_of(a.vocab);
  Part* p = static_cast<Part*>(a.workspace);
  Part* q = a.draft ? p + (int64_t)rows * chunks : nullptr;
  const Sizes z = {chunks, p, q, a.draft ? reinterpret_cast<double*>(q + (int64_t)rows * chunks) : nullptr};
  verify_rows_kernel<<<dim3((unsigned)((int64_t)rows * (a.draft ? 2 : 1) * chunks)), kThreads, 0, stream>>>(a, z);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.draft) {
    verify_rest_kernel<<<dim3((unsigned)((int64_t)a.B * chunks)), kThreads, 0, stream>>>(a, z);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  verify_draw_kernel<<<dim3((unsigned)a.B), kThreads, 0, stream>>>(a, z);
  return hipGetLastError();
}

}  // namespace nvfp4

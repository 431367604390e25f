// Gated linear attention with the delta rule over prompts, in chunks of 64 tokens.
//
// Within a chunk, with G_t the sum of the log decays up to token t, S the state
// before the chunk and rows as matrices,
//   A_ij = beta_i (k_i . k_j) e^(G_i - G_j)  (i > j),   T = (1 + A)^-1 diag(beta),
//   N = T (V - e^G K S)                       (the values that are written; N = V without beta),
//   O = scale (e^G Q S + P N),  P_ij = (q_i . k_j) e^(G_i - G_j)  (i >= j),
//   S' = e^(G_64) S + K^T (e^(G_64 - G) N).
// Two kernels: the first computes T and P of every chunk at once, the second
// carries the state from chunk to chunk, a workgroup for 16, 32 or 64 of its columns, or
// for 128 where there are heads enough; columns touch no other column.  Bound by the latency of that chain: 8192 tokens of 32
// heads of 128 x 128 take 244 us, of which the first kernel is 48 and 128 chunks one
// after the other, at 1.5 us (three exchanges through LDS and their barriers), the rest.
// Without beta also by memory: 6 of up to 8192 take 411 us, 88 of them the first kernel, and
// move 1434 MB for a call of 663 (P out and in, keys and queries for each kernel and each slab
// of columns), 280 us at a copy's rate.
//
// Precision.  The state is binary32 and its path keeps binary32's accuracy on the
// bf16 matrix cores (fp32 matrix products run at 1/16 of their rate): q, k and v are
// bf16 already, and a binary32 operand x enters as three bf16 planes, x = hi + mid +
// lo to 24 significant bits, so K S is three products, and T times a binary32
// matrix the six of the nine plane products that are above 2^-24.  What only
// reaches the bf16 output keeps two planes (16 bits).  Sums accumulate in binary32.
// G is summed in binary64, so that differences of far decays keep their digits.
#include <limits.h>

#include <algorithm>

#include "common.hpp"
#include "mixers.hpp"
#include "mixers_device.hpp"

namespace nvfp4 {

constexpr int kChunk = 64;

// Workspace of one (chunk, value head): operand blocks of 1 KB, lane-contiguous --
// block (i, s) of a matrix holds for lane (t, g) row 16 i + t, columns 32 s + 4 g + j
// and 32 s + 16 + 4 g + j (j < 4) -- for the six blocks that a lower triangle
// touches, T in three planes and P in two; then e^G and e^(G_64 - G) of the rows.
constexpr int kBlocks = 6, kBlockBytes = 1024;
constexpr int kTPlanes = 3, kPPlanes = 2;
__host__ __device__ constexpr int block_of(int i, int s) { return s == 0 ? i : 2 + i; }  // s == 1: i is 2 or 3
struct Slot {
  static constexpr int kP = 0, kDecay = kP + kBlocks * kPPlanes * kBlockBytes, kLeft = kDecay + kChunk * 4,
                       kT = kDecay + 1024, kBytesLinear = kT, kBytesDelta = kT + kBlocks * kTPlanes * kBlockBytes;
};

// Chunk slots: sequence b's chunks start at cu[b] / 64 + b, so no two share one.
__host__ __device__ inline int64_t chunk_slots(int64_t T, int64_t B) { return T / kChunk + B; }

// Two binary32 values as N bf16 planes: what a plane leaves goes to the next.
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&out)[N]) {
#pragma unroll
  for (int p = 0; p < N; ++p) {
    out[p] = bf16_pair(a, b);
    a -= __uint_as_float(out[p] << 16);
    b -= __uint_as_float(out[p] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float4_t mfma_bf16(uint4 a, uint4 b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ float4_t mfma_bf16_16(uint2 a, uint2 b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4_t, a), __builtin_bit_cast(short4_t, b), c, 0,
                                                   0, 0);
}

struct Rows {
  int64_t first;  // row of the sequence's first token
  int count;
};
__device__ __forceinline__ Rows rows_of(const GdnArgs& a, int b) {
  // the same in every lane: held in scalar registers, with the addresses that follow from them
  const int64_t lo = __builtin_amdgcn_readfirstlane(a.cu[b]), hi = __builtin_amdgcn_readfirstlane(a.cu[b + 1]);
  const int64_t first = min(max(lo, (int64_t)0), a.T);
  return {first, (int)(min(max(hi, first), a.T) - first)};
}

// The sequence that is r-th by length, longest first: workgroups start in turn, and a
// long sequence that starts late is waited for alone.  (Every order is right; beyond
// 64 sequences their own is taken.)
__device__ __forceinline__ int by_length(const GdnArgs& a, int r) {
  if (a.B > 64) return r;
  const int lane = threadIdx.x % 64;
  const int mine = lane < a.B ? a.cu[lane + 1] - a.cu[lane] : INT_MIN;
  int rank = 0;
  for (int i = 0; i < (int)a.B; ++i) {
    const int other = __builtin_amdgcn_readlane(mine, i);
    rank += other > mine || (other == mine && i < lane) ? 1 : 0;
  }
  return __ffsll((unsigned long long)__ballot(lane < a.B && rank == r)) - 1;
}

// Whether a sequence has more than one and a half times a CU's fair share of the work of a
// launch of whole heads: alone it would outlast the rest (see launch_prefill).
__device__ __forceinline__ bool is_long(const GdnArgs& a, int count) {
  return (int64_t)count * (2 * kCUs) > 3 * a.T * a.v_heads * (a.v_dim / 128);
}

// The r-th of the long sequences; -1 if there are fewer.
__device__ __forceinline__ int long_sequence(const GdnArgs& a, int r) {
  const int lane = threadIdx.x % 64;
  for (int64_t b0 = 0; b0 < a.B; b0 += 64) {
    const int64_t b = b0 + lane;
    int count = 0;
    if (b < a.B) {
      const int64_t first = min(max((int64_t)a.cu[b], (int64_t)0), a.T);
      count = (int)(min(max((int64_t)a.cu[b + 1], first), a.T) - first);
    }
    unsigned long long found = __ballot(is_long(a, count));
    if (r >= __popcll(found)) {
      r -= __popcll(found);
      continue;
    }
    for (; r > 0; --r) found &= found - 1;
    return (int)b0 + __ffsll(found) - 1;
  }
  return -1;
}

// ---- T and P of every chunk ------------------------------------------------------
// A workgroup takes one chunk of one value head; wave w holds rows 16 w .. 16 w + 15 of
// K K^T and Q K^T.  The inverse: the four 16 x 16 diagonal blocks by substitution,
// all at once in one wave (lane (n, g): column n of block g), then the blocks below
// them, T_ij = -T_ii sum_k A_ik T_kj, one diagonal after the other, as fp32 matrix
// products.  A wave's rows of P and T become operand blocks through LDS rows that no
// other wave touches meanwhile.
constexpr int kLd = 68;  // row stride of the 64 x 64 matrices in LDS
constexpr float kLog2e = 1.44269504088896340736f;

// e^x of a sum of log decays (x <= 0).  The cast, the constant and the product are off by 1, 0.23
// and 1 times 2^-24 relative, so the exponent by 2.23 2^-24 |x|; |x| e^x is at most 0.37, so
// the factor by 0.83 2^-24 of its largest value, 1, and by the exponential's own 2^-23 of itself.
__device__ __forceinline__ float fade_of(double x) { return __builtin_amdgcn_exp2f((float)x * kLog2e); }

// Four rows' columns 32 s + 4 g + 0 .. 3 and 32 s + 16 + 4 g + 0 .. 3 as operand planes at `to`.
template <int P>
__device__ __forceinline__ void put_block(uint8_t* to, int blk, int lane, float4_t x, float4_t y) {
  uint32_t z[4][P];
  split_pair(x[0], x[1], z[0]);
  split_pair(x[2], x[3], z[1]);
  split_pair(y[0], y[1], z[2]);
  split_pair(y[2], y[3], z[3]);
#pragma unroll
  for (int p = 0; p < P; ++p)
    *reinterpret_cast<uint4*>(to + (p * kBlocks + blk) * kBlockBytes + lane * 16) =
        make_uint4(z[0][p], z[1][p], z[2][p], z[3][p]);
}

template <int DK, bool DELTA>
__global__ __launch_bounds__(256, 4) void gdn_chunk_kernel(GdnArgs a) {
  constexpr int kRow = DK * 2 + 16, kPieces = DK / 8, kLoads = kChunk * kPieces / 256;
  static_assert(kChunk * kRow <= kChunk * kLd * 4, "key and query rows lie where the matrices come");
  __shared__ __align__(16) float mat[kChunk * kLd], inv[kChunk * kLd];
  __shared__ double sums[kChunk];
  __shared__ __align__(16) float betas[kChunk];
  const int lane = threadIdx.x % 64, n = lane % 16, g = lane / 16;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // the value heads of a key head run one after the other on one XCD (workgroups go round
  // the eight in turn), so that its L2 has the keys and queries for all but the first
  // (two value heads to a key head: 48 us against 57, without beta 86 against 98)
  const int group = a.v_heads / a.k_heads, hk = blockIdx.y, hv = hk * group + blockIdx.x / 8 % group;
  const int64_t slot = (int64_t)(blockIdx.x / 8 / group) * 8 + blockIdx.x % 8;
  // the sequence whose slots this chunk's index falls into
  int b = -1;
  for (int64_t b0 = 0; b0 < a.B; b0 += 64) {
    const int64_t i = b0 + lane;
    const bool before = i < a.B && min(max((int64_t)a.cu[i], (int64_t)0), a.T) / kChunk + i <= slot;
    b += __popcll(__ballot(before));
  }
  if (b < 0) return;
  const Rows rows = rows_of(a, b);
  const int chunk = (int)(slot - (rows.first / kChunk + b));
  const int count = min(kChunk, rows.count - chunk * kChunk);
  if (chunk < 0 || count <= 0) return;
  const int64_t row0 = rows.first + (int64_t)chunk * kChunk;
  uint8_t* to = static_cast<uint8_t*>(a.workspace) +
                (slot * a.v_heads + hv) * (int64_t)(DELTA ? Slot::kBytesDelta : Slot::kBytesLinear);

  uint8_t* keys = reinterpret_cast<uint8_t*>(mat);
  uint8_t* queries = reinterpret_cast<uint8_t*>(inv);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (i * 256 + (int)threadIdx.x) / kPieces, c = threadIdx.x % kPieces;
    const int64_t from = row0 + min(r, count - 1);
    *reinterpret_cast<u32x4_t*>(keys + r * kRow + c * 16) =
        *reinterpret_cast<const u32x4_t*>(a.k + from * a.ldk + hk * DK + c * 8);
    *reinterpret_cast<u32x4_t*>(queries + r * kRow + c * 16) =
        *reinterpret_cast<const u32x4_t*>(a.q + from * a.ldq + hk * DK + c * 8);
  }
  if (w == 0) {
    const int64_t r = row0 + min(lane, count - 1);
    // below -1000 a factor is 0 in binary32 either way, and the sums stay finite
    const float step = lane < count ? a.g[r * a.ldg + hv] : 0.0f;
    double sum = step < -1000.0f ? -1000.0 : (double)step;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double x = __shfl_up(sum, d);
      if (lane >= d) sum += x;
    }
    sums[lane] = sum;
    betas[lane] = DELTA && lane < count ? a.beta[r * a.ldb + hv] : 0.0f;
    const double all = __shfl(sum, 63);
    reinterpret_cast<float*>(to + Slot::kDecay)[lane] = fade_of(sum);
    reinterpret_cast<float*>(to + Slot::kLeft)[lane] = lane < count ? fade_of(all - sum) : 0.0f;
  }
  __syncthreads();

  // rows 16 w + .. of K K^T and Q K^T against column blocks 0 .. w
  float4_t kk[4], qk[4];
  {
    uint4 ka[DK / 32], qa[DK / 32];
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      ka[s] = *reinterpret_cast<const uint4*>(keys + (16 * w + n) * kRow + s * 64 + g * 16);
      qa[s] = *reinterpret_cast<const uint4*>(queries + (16 * w + n) * kRow + s * 64 + g * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      kk[j] = qk[j] = {0, 0, 0, 0};
      if (j > w) continue;
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const uint4 kb = *reinterpret_cast<const uint4*>(keys + (16 * j + n) * kRow + s * 64 + g * 16);
        if (DELTA) kk[j] = mfma_bf16(ka[s], kb, kk[j]);
        qk[j] = mfma_bf16(qa[s], kb, qk[j]);
      }
    }
  }
  __syncthreads();
  // P through this wave's rows, then A into them
  double mine[4];
  float beta[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    mine[r] = sums[16 * w + 4 * g + r];
    beta[r] = betas[16 * w + 4 * g + r];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j / 2 > w / 2) continue;  // (a step's second half may lie above the diagonal: zeros)
    const int col = 16 * j + n;
    const double theirs = sums[col];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      const float fade = row >= col && row < count ? fade_of(mine[r] - theirs) : 0.0f;
      mat[row * kLd + col] = fade != 0.0f ? a.scale * qk[j][r] * fade : 0.0f;
      kk[j][r] = row > col && fade != 0.0f ? beta[r] * kk[j][r] * fade : 0.0f;
    }
  }
  wave_lds_fence();
  const int at = (16 * w + n) * kLd + 4 * g;
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (s <= w / 2)
      put_block<kPPlanes>(to + Slot::kP, block_of(w, s), lane, *reinterpret_cast<const float4_t*>(mat + at + 32 * s),
                          *reinterpret_cast<const float4_t*>(mat + at + 32 * s + 16));
  if (!DELTA) return;
  wave_lds_fence();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j / 2 > w / 2) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      mat[(16 * w + 4 * g + r) * kLd + 16 * j + n] = kk[j][r];
      if (j > w) inv[(16 * w + 4 * g + r) * kLd + 16 * j + n] = 0.0f;
    }
  }
  __syncthreads();
  if (w == 0) {  // column n of the inverse of diagonal block g
    const float* blk = mat + (16 * g) * kLd + 16 * g;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const float4_t l = *reinterpret_cast<const float4_t*>(blk + i * kLd + j);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) s = __builtin_fmaf(-l[e], x[j + e], s);
      }
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) inv[(16 * g + i) * kLd + 16 * g + n] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < 4; ++d) {  // blocks (w, w - d)
    const int j = w - d;
    if (j >= 0) {
      float4_t m = {0, 0, 0, 0}, t = {0, 0, 0, 0};
      for (int k = j; k < w; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          m = __builtin_amdgcn_mfma_f32_16x16x4f32(mat[(16 * w + n) * kLd + 16 * k + 4 * s + g],
                                                   inv[(16 * k + 4 * s + g) * kLd + 16 * j + n], m, 0, 0, 0);
      // rows 4 g + r of m are where step r of the next product wants them
#pragma unroll
      for (int r = 0; r < 4; ++r)
        t = __builtin_amdgcn_mfma_f32_16x16x4f32(inv[(16 * w + n) * kLd + 16 * w + 4 * g + r], m[r], t, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) inv[(16 * w + 4 * g + r) * kLd + 16 * j + n] = -t[r];
    }
    if (d < 3) __syncthreads();
  }
  wave_lds_fence();
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (s <= w / 2)
      put_block<kTPlanes>(to + Slot::kT, block_of(w, s), lane,
                          *reinterpret_cast<const float4_t*>(inv + at + 32 * s) *
                              *reinterpret_cast<const float4_t*>(betas + 32 * s + 4 * g),
                          *reinterpret_cast<const float4_t*>(inv + at + 32 * s + 16) *
                              *reinterpret_cast<const float4_t*>(betas + 32 * s + 16 + 4 * g));
}

// ---- the state from chunk to chunk -----------------------------------------------
// A workgroup of twelve waves carries 16 NT columns: four for the chain from state to
// state, four for the outputs and four that feed the chain, which fill its waits on
// the same SIMDs.
//
// Chain wave w owns a quarter of the state's rows, in registers throughout: a
// product leaves row 4 g + r in register r, which is how the next product's right
// operand wants its rows, so the state's planes are right operands as they are,
// with the left operand's columns taken in that order.  Its products with the
// wave's quarter of the key columns are shares of K S for all 64 tokens, which the
// four waves add up through LDS, each for 16 tokens; R = V - e^G K S and N = T R pass
// between the waves as planes in operand order (16 bytes for each lane, no bank
// conflicts), and the update needs the wave's quarter of K^T only.  Output wave w
// takes tokens 16 w .. 16 w + 15 of Q S and P N.  Without beta N is V, known before
// the chunk.
//
// Each area of LDS is written between one pair of barriers and read between the next.
template <int DK, int NT, bool DELTA>
struct StateLds {
  static constexpr int kRun = DK / 4 * 2;                           // bytes of a wave's quarter of a key row
  static constexpr int kKeyRow = kRun + 16;                         // rows fall on different banks
  static constexpr int kTurned = DK / 64 * 2;                       // operand blocks of a wave's rows of K^T
  static constexpr int kS = 0;                                      // two planes of S, for the outputs
  static constexpr int kN = kS + 2 * (DK / 32) * NT * 1024;         // planes of e^(G_64 - G) N, then of N
  static constexpr int kOut = 6 * NT * 1024;                        // of the latter in kN
  static constexpr int kR = kN + kOut + (DELTA ? 2 : 1) * 2 * NT * 1024;
  static constexpr int kShares = kR + (DELTA ? 6 * NT * 1024 : 0);  // of K S: [token tile][column tile][wave]
  static constexpr int kKeys = kShares + (DELTA ? 16 * NT * 1024 : 0);
  static constexpr int kKeysT = kKeys + 4 * kChunk * kKeyRow;
  // values and decays of the 16 tokens of a wave pair; an output wave's results and queries
  static constexpr int kRow = 32 * NT + 16;
  static constexpr int kValues = kKeysT + 4 * kTurned * 1024;
  static constexpr int kDecays = kValues + 4 * 16 * kRow;           // e^G, e^(G_64 - G), e^(G_64)
  static constexpr int kResults = kDecays + 4 * 144;
  static constexpr int kQueryRow = DK * 2 + 16;
  static constexpr int kQueries = kResults + 4 * 16 * kRow;
  static constexpr int kBytes = kQueries + 4 * 16 * kQueryRow;
};

// What both halves of the workgroup share.
template <int DK, int NT, bool DELTA>
struct StateWave {
  using L = StateLds<DK, NT, DELTA>;
  static constexpr int TW = DK / 64;
  const GdnArgs& a;
  uint8_t* lds;
  int64_t first;     // row of the sequence's first token
  int count, chunks; // its tokens and chunks
  int hk, col;       // key head; first column of the rows of v and out
  const uint8_t* ws; // the first chunk's slot
  int64_t ws_step;
  int w, lane, n, g;

  __device__ __forceinline__ int last_of(int ch) const { return min(kChunk, count - ch * kChunk) - 1; }
  __device__ __forceinline__ uint4 get(const uint8_t* x, int p, int per, int s, int c) const {
    return *reinterpret_cast<const uint4*>(x + ((p * per + s) * NT + c) * 1024 + lane * 16);
  }
  // 8 elements of step s of a q row in LDS, in the order of the state's planes
  __device__ __forceinline__ uint4 run(const uint16_t* row, int s) const {
    if constexpr (TW == 2) return *reinterpret_cast<const uint4*>(row + 32 * s + 8 * g);
    const uint2 x = *reinterpret_cast<const uint2*>(row + 32 * s + 4 * g);
    const uint2 y = *reinterpret_cast<const uint2*>(row + 32 * s + 16 + 4 * g);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  // block (w, s) of a matrix's plane in chunk ch's slot
  __device__ __forceinline__ uint4 block(int ch, int at, int p, int s) const {
    return *reinterpret_cast<const uint4*>(ws + ch * ws_step + at + (p * kBlocks + block_of(w, s)) * kBlockBytes + lane * 16);
  }
  // four rows of this wave as P planes at x
  template <int P>
  __device__ __forceinline__ void put_rows(uint8_t* x, int c, float4_t v) const {
    uint32_t z[2][P];
    split_pair(v[0], v[1], z[0]);
    split_pair(v[2], v[3], z[1]);
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<uint2*>(x + ((p * 2 + w / 2) * NT + c) * 1024 + lane * 16 + (w % 2) * 8) =
          make_uint2(z[0][p], z[1][p]);
  }
};

// Rows of a tensor that a lane reads or writes in chunk after chunk: N pointers, moved on by
// a chunk's rows.
template <int N, typename T>
struct RowPointers {
  T* p[N];
  __device__ __forceinline__ void on(int64_t step) {
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] += step;
  }
};

template <int DK, int NT, bool DELTA>
__device__ __forceinline__ void carry_state(const StateWave<DK, NT, DELTA>& m, float* st, bool load) {
  using L = StateLds<DK, NT, DELTA>;
  constexpr int TW = DK / 64;  // state tiles, and dwords of a lane's piece of a key row by two
  const GdnArgs& a = m.a;
  const int w = m.w, n = m.n, g = m.g, lane = m.lane, chunks = m.chunks;
  const int steps = w / 2 + 1;  // 32-token steps that rows 16 w .. reach in a lower triangle
  // tile i, register r: state row w DK / 4 + (4 g + r) TW + i
  float4_t S[NT][TW];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[c][i][r] = load ? st[(int64_t)(r * TW + i) * a.v_dim + 16 * c] : 0.0f;

  const uint8_t* keys = m.lds + L::kKeys + w * kChunk * L::kKeyRow;
  const uint8_t* values = m.lds + L::kValues + w * 16 * L::kRow;
  const uint8_t* decays = m.lds + L::kDecays + w * 144;
  uint4 ta[2][3];
  uint32_t ka[4][2 * TW];  // left operand of K S: 4 TW elements of the key rows of tokens 16 i + n
  auto get_keys = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* from = keys + (16 * i + n) * L::kKeyRow + g * 8 * TW;
      if constexpr (TW == 2) {
        const uint4 y = *reinterpret_cast<const uint4*>(from);
        ka[i][0] = y.x, ka[i][1] = y.y, ka[i][2] = y.z, ka[i][3] = y.w;
      } else {
        const uint2 y = *reinterpret_cast<const uint2*>(from);
        ka[i][0] = y.x, ka[i][1] = y.y;
      }
    }
  };
  auto fetch_t = [&](int ch) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        if (s < steps) ta[s][p] = m.block(ch, Slot::kT, p, s);
  };
  if (chunks > 0) {
    if (DELTA) fetch_t(0);
    __syncthreads();
  }
  for (int ch = 0; ch < chunks; ++ch) {
    const int next = min(ch + 1, chunks - 1);
    if (DELTA) get_keys();
    // shares of K S from this wave's rows of S; two planes of S for the outputs
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      uint32_t z[2 * TW][DELTA ? 3 : 2];
#pragma unroll
      for (int e = 0; e < 2 * TW; ++e) {
        const int f = 2 * e;
        split_pair(S[c][f % TW][f / TW], S[c][(f + 1) % TW][(f + 1) / TW], z[e]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if constexpr (TW == 2)
          *reinterpret_cast<uint4*>(m.lds + L::kS + ((p * (DK / 32) + w) * NT + c) * 1024 + lane * 16) =
              make_uint4(z[0][p], z[1][p], z[2][p], z[3][p]);
        else
          *reinterpret_cast<uint2*>(m.lds + L::kS + ((p * (DK / 32) + w / 2) * NT + c) * 1024 + lane * 16 + (w % 2) * 8) =
              make_uint2(z[0][p], z[1][p]);
      }
      if (DELTA) {
        float4_t ks[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = {0, 0, 0, 0};
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            constexpr int P = DELTA ? 3 : 2;
            if constexpr (TW == 2)
              ks[i] = mfma_bf16(make_uint4(ka[i][0], ka[i][1], ka[i][2], ka[i][3]),
                                make_uint4(z[0][p % P], z[1][p % P], z[2][p % P], z[3][p % P]), ks[i]);
            else
              ks[i] = mfma_bf16_16(make_uint2(ka[i][0], ka[i][1]), make_uint2(z[0][p % P], z[1][p % P]), ks[i]);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4_t*>(m.lds + L::kShares + ((i * NT + c) * 4 + w) * 1024 + lane * 16) = ks[i];
      }
    }
    __syncthreads();
    const float4_t decay = *reinterpret_cast<const float4_t*>(decays + 16 * g);
    const float4_t left = *reinterpret_cast<const float4_t*>(decays + 64 + 16 * g);
    const float whole = *reinterpret_cast<const float*>(decays + 128);
    float4_t N[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        N[c][r] = __uint_as_float(
            (uint32_t) * reinterpret_cast<const uint16_t*>(values + (4 * g + r) * L::kRow + (16 * c + n) * 2) << 16);
      if (DELTA) {  // R = V - e^G K S
        float4_t sh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sh[i] = *reinterpret_cast<const float4_t*>(m.lds + L::kShares + ((w * NT + c) * 4 + i) * 1024 + lane * 16);
        N[c] -= decay * ((sh[0] + sh[1]) + (sh[2] + sh[3]));
        m.template put_rows<3>(m.lds + L::kR, c, N[c]);
      } else {
        m.template put_rows<3>(m.lds + L::kN, c, N[c] * left);
        m.template put_rows<1>(m.lds + L::kN + L::kOut, c, N[c]);
      }
    }
    uint4 kt[2][TW];
    auto get_turned = [&] {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < TW; ++i)
          kt[s][i] = *reinterpret_cast<const uint4*>(m.lds + L::kKeysT + (w * L::kTurned + s * TW + i) * 1024 + lane * 16);
    };
    if (!DELTA) get_turned();  // before the chunk's last barrier: then the next chunk's are put there
    __syncthreads();
    if (DELTA) get_turned();
    if (DELTA) {  // N = T R
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        float4_t acc[3] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s >= steps) continue;
          const uint8_t* y = m.lds + L::kR;
          const uint4 r0 = m.get(y, 0, 2, s, c), r1 = m.get(y, 1, 2, s, c), r2 = m.get(y, 2, 2, s, c);
          acc[0] = mfma_bf16(ta[s][0], r0, acc[0]);
          acc[1] = mfma_bf16(ta[s][1], r0, acc[1]);
          acc[2] = mfma_bf16(ta[s][2], r0, acc[2]);
          acc[1] = mfma_bf16(ta[s][0], r1, acc[1]);
          acc[2] = mfma_bf16(ta[s][1], r1, acc[2]);
          acc[2] = mfma_bf16(ta[s][0], r2, acc[2]);
        }
        N[c] = (acc[2] + acc[1]) + acc[0];
        m.template put_rows<3>(m.lds + L::kN, c, N[c] * left);
        m.template put_rows<2>(m.lds + L::kN + L::kOut, c, N[c]);
      }
      fetch_t(next);
      __syncthreads();
    }
    // S' = e^G S + K^T (e^(G_64 - G) N)
#pragma unroll
    for (int c = 0; c < NT; ++c) {
#pragma unroll
      for (int i = 0; i < TW; ++i) S[c][i] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 2; p >= 0; --p) {
          const uint4 u = m.get(m.lds + L::kN, p, 2, s, c);
#pragma unroll
          for (int i = 0; i < TW; ++i) S[c][i] = mfma_bf16(kt[s][i], u, S[c][i]);
        }
    }
  }
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) st[(int64_t)(r * TW + i) * a.v_dim + 16 * c] = S[c][i][r];
}

// What comes from memory is fetched two chunks ahead as rows in pieces of 16 bytes,
// lanes side by side along a row, and the decays one to a lane, and sorted through
// LDS.  (A load in operand order, 16 rows side by side, takes one turn of the vector
// cache for each lane, four times as many; a load of 2 bytes a lane as many as one
// of 16.)
//
// Feeding wave w: the chain's left operands, w's quarter of the key rows as they
// are and transposed, its 16 rows of values and its decays.
template <int DK, int NT, bool DELTA>
__device__ __forceinline__ void feed_chain(const StateWave<DK, NT, DELTA>& m) {
  using L = StateLds<DK, NT, DELTA>;
  constexpr int TW = DK / 64;
  constexpr int kPieces = L::kRun / 16, kLoads = kChunk * kPieces / 64;  // of a key row; of a lane
  constexpr int kValuePieces = 2 * NT, kValueLoads = (32 * NT + 63) / 64;  // of a row of values; of a lane
  const GdnArgs& a = m.a;
  const int w = m.w, n = m.n, g = m.g, lane = m.lane, chunks = m.chunks;
  RowPointers<kLoads, const uint16_t> kp;
  RowPointers<kValueLoads, const uint16_t> vp;
  struct Fetched {
    u32x4_t k[kLoads], v[kValueLoads];
    float decay;
  };
  Fetched even, odd;
  uint4 kt[2][TW];
  uint8_t* keys = m.lds + L::kKeys + w * kChunk * L::kKeyRow;
  const bool has_piece = lane < 32 * NT;
  const int v_row = lane / kValuePieces % 16, v_piece = lane % kValuePieces;
  const int decay_at = lane < 16 ? Slot::kDecay + (16 * w + n) * 4
                                 : (lane < 32 ? Slot::kLeft + (16 * w + n) * 4 : Slot::kDecay + 63 * 4);
  auto point = [&](int ch) {
    const int64_t row0 = m.first + (int64_t)ch * kChunk;
    const int last = m.last_of(ch);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      kp.p[i] = a.k + (row0 + min((i * 64 + lane) / kPieces, last)) * a.ldk + m.hk * DK + w * (DK / 4) + lane % kPieces * 8;
#pragma unroll
    for (int i = 0; i < kValueLoads; ++i)
      vp.p[i] = a.v + m.col + 8 * v_piece + (row0 + min(16 * w + i * (64 / kValuePieces) + v_row, last)) * a.ldv;
  };
  auto fetch = [&](Fetched& x, int ch) {  // where the pointers stand
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x.k[i] = *reinterpret_cast<const u32x4_t*>(kp.p[i]);
#pragma unroll
    for (int i = 0; i < kValueLoads; ++i)
      if (has_piece) x.v[i] = *reinterpret_cast<const u32x4_t*>(vp.p[i]);
    x.decay = *reinterpret_cast<const float*>(m.ws + ch * m.ws_step + decay_at);
  };
  auto put_keys = [&](const Fetched& x) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<u32x4_t*>(keys + (i * 64 + lane) / kPieces * L::kKeyRow + lane % kPieces * 16) = x.k[i];
  };
  // the wave's rows of K^T: TW elements of 8 tokens' rows, transposed within the lane
  auto turn_keys = [&] {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* from = keys + (32 * s + (j / 4) * 16 + 4 * g + j % 4) * L::kKeyRow + n * TW * 2;
        if constexpr (TW == 2)
          z[j] = *reinterpret_cast<const uint32_t*>(from);
        else
          z[j] = *reinterpret_cast<const uint16_t*>(from);
      }
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          e[j] = i ? high_halves(z[2 * j], z[2 * j + 1]) : low_halves(z[2 * j], z[2 * j + 1]);
        kt[s][i] = make_uint4(e[0], e[1], e[2], e[3]);
      }
    }
  };
  auto put_rest = [&](const Fetched& x) {  // K^T, values and decays, once the chain has read those of the chunk before
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < TW; ++i)
        *reinterpret_cast<uint4*>(m.lds + L::kKeysT + (w * L::kTurned + s * TW + i) * 1024 + lane * 16) = kt[s][i];
#pragma unroll
    for (int i = 0; i < kValueLoads; ++i)
      if (has_piece)
        *reinterpret_cast<u32x4_t*>(m.lds + L::kValues + (w * 16 + i * (64 / kValuePieces) + v_row) * L::kRow +
                                    16 * v_piece) = x.v[i];
    if (lane <= 32) reinterpret_cast<float*>(m.lds + L::kDecays + w * 144)[lane] = x.decay;
  };
  auto on = [&](int from) {  // the pointers to the next chunk, or to the last one again
    const int to = min(from + 1, chunks - 1);
    if (m.last_of(to) == kChunk - 1) {
      if (to > from) kp.on(a.ldk * kChunk), vp.on(a.ldv * kChunk);
    } else {
      point(to);
    }
    return to;
  };
  if (chunks == 0) return;
  point(0);
  fetch(even, 0);
  int at = on(0);  // where the pointers stand
  fetch(odd, at);
  put_keys(even);
  wave_lds_fence();
  turn_keys();
  put_rest(even);
  at = on(at);
  fetch(even, at);
  __syncthreads();
  auto chunk = [&](Fetched& next) {  // behind the last chunk, its own again
    __syncthreads();
    __syncthreads();
    put_keys(next);
    wave_lds_fence();
    turn_keys();
    if (DELTA) __syncthreads();
    put_rest(next);
    at = on(at);
    fetch(next, at);
  };
  for (int ch = 0; ch < chunks; ch += 2) {
    chunk(odd);
    if (ch + 1 < chunks) chunk(even);
  }
}

// Output wave w: tokens 16 w .. 16 w + 15.
template <int DK, int NT, bool DELTA>
__device__ __forceinline__ void write_outputs(const StateWave<DK, NT, DELTA>& m) {
  using L = StateLds<DK, NT, DELTA>;
  constexpr int KS = DK / 32;
  constexpr int kPieces = DK / 8, kLoads = 16 * kPieces / 64;  // of a query row; of a lane
  const GdnArgs& a = m.a;
  const int w = m.w, n = m.n, g = m.g, lane = m.lane, chunks = m.chunks;
  const int steps = w / 2 + 1;
  RowPointers<kLoads, const uint16_t> qp;
  constexpr int kOutPieces = 2 * NT, kOutStores = (32 * NT + 63) / 64;  // of a row of results; of a lane
  RowPointers<kOutStores, uint16_t> op;
  struct Fetched {
    u32x4_t q[kLoads];
  };
  Fetched even, odd;
  uint4 qa[KS], pa[2][2];
  uint8_t* queries = m.lds + L::kQueries + w * 16 * L::kQueryRow;
  uint8_t* results = m.lds + L::kResults + w * 16 * L::kRow;
  const int o_row = lane / kOutPieces % 16, o_piece = lane % kOutPieces;
  auto point = [&](int ch) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      qp.p[i] = a.q + (m.first + (int64_t)ch * kChunk + min(16 * w + (i * 64 + lane) / kPieces, m.last_of(ch))) * a.ldq +
                m.hk * DK + lane % kPieces * 8;
  };
  auto fetch_q = [&](Fetched& x) {  // where the pointers stand
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x.q[i] = *reinterpret_cast<const u32x4_t*>(qp.p[i]);
  };
  auto fetch_p = [&](int ch) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (s < steps) pa[s][p] = m.block(ch, Slot::kP, p, s);
  };
  auto sort_queries = [&](const Fetched& x) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<u32x4_t*>(queries + (i * 64 + lane) / kPieces * L::kQueryRow + lane % kPieces * 16) = x.q[i];
    wave_lds_fence();
#pragma unroll
    for (int s = 0; s < KS; ++s) qa[s] = m.run(reinterpret_cast<const uint16_t*>(queries + n * L::kQueryRow), s);
  };
  auto on = [&](int from) {
    const int to = min(from + 1, chunks - 1);
    if (m.last_of(to) == kChunk - 1) {
      if (to > from) qp.on(a.ldq * kChunk);
    } else {
      point(to);
    }
    return to;
  };
  if (chunks == 0) return;
  point(0);
#pragma unroll
  for (int i = 0; i < kOutStores; ++i)
    op.p[i] = a.out + m.col + 8 * o_piece + (m.first + 16 * w + i * (64 / kOutPieces) + o_row) * a.ldo;
  fetch_q(even);
  fetch_p(0);
  int at = on(0);  // where the pointers stand
  fetch_q(odd);
  sort_queries(even);
  at = on(at);
  fetch_q(even);
  __syncthreads();
  auto chunk = [&](int ch, Fetched& next) {
    const int last = m.last_of(ch);
    __syncthreads();
    const float4_t decay = *reinterpret_cast<const float4_t*>(m.lds + L::kDecays + w * 144 + 16 * g);
    float4_t o[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      float4_t lo = {0, 0, 0, 0};
      o[c] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        o[c] = mfma_bf16(qa[s], m.get(m.lds + L::kS, 0, KS, s, c), o[c]);
        lo = mfma_bf16(qa[s], m.get(m.lds + L::kS, 1, KS, s, c), lo);
      }
      o[c] = (o[c] + lo) * (decay * a.scale);
    }
    __syncthreads();
    sort_queries(next);  // behind the last chunk, its own again
    at = on(at);
    fetch_q(next);
    if (DELTA) __syncthreads();
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      float4_t lo = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s >= steps) continue;
        const uint4 n0 = m.get(m.lds + L::kN + L::kOut, 0, 2, s, c);
        o[c] = mfma_bf16(pa[s][0], n0, o[c]);
        lo = mfma_bf16(pa[s][1], n0, lo);
        if (DELTA) lo = mfma_bf16(pa[s][0], m.get(m.lds + L::kN + L::kOut, 1, 2, s, c), lo);
      }
      o[c] += lo;
    }
    fetch_p(min(ch + 1, chunks - 1));
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<uint16_t*>(results + (4 * g + r) * L::kRow + (16 * c + n) * 2) =
            __builtin_bit_cast(uint16_t, (__bf16)o[c][r]);
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < kOutStores; ++i) {
      const int row = i * (64 / kOutPieces) + o_row;
      if (lane < 32 * NT && 16 * w + row <= last)
        *reinterpret_cast<uint4*>(op.p[i]) = *reinterpret_cast<const uint4*>(results + row * L::kRow + 16 * o_piece);
    }
    op.on(a.ldo * kChunk);
  };
  for (int ch = 0; ch < chunks; ch += 2) {
    chunk(ch, odd);
    if (ch + 1 < chunks) chunk(ch + 1, even);
  }
}

template <int DK, int NT, bool DELTA>
__global__ __launch_bounds__(768, 3) void gdn_state_kernel(GdnArgs a, bool long_only) {
  using L = StateLds<DK, NT, DELTA>;
  __shared__ __align__(16) uint8_t lds[L::kBytes];
  const int slabs = a.v_dim / (16 * NT);
  // slabs of a head run on one XCD (workgroups go round the eight in turn) and share its L2
  const int64_t turn = blockIdx.x / 8;
  const int64_t pair = (turn / slabs) * 8 + blockIdx.x % 8;
  const int slab = (int)(turn % slabs);
  if (pair >= a.B * a.v_heads) return;
  const int r = (int)(pair / a.v_heads), b = long_only ? long_sequence(a, r) : by_length(a, r), h = (int)(pair % a.v_heads);
  if (b < 0) return;
  const int64_t slot = a.index ? __builtin_amdgcn_readfirstlane(a.index[b]) : b;
  if (slot < 0 || slot >= a.num_states) return;
  const int lane = threadIdx.x % 64, n = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), w = wave % 4;
  const Rows rows = rows_of(a, b);
  const int64_t step = (int64_t)a.v_heads * (DELTA ? Slot::kBytesDelta : Slot::kBytesLinear);
  const uint8_t* ws = static_cast<const uint8_t*>(a.workspace) + (rows.first / kChunk + b) * step +
                      h * (int64_t)(DELTA ? Slot::kBytesDelta : Slot::kBytesLinear);
  const StateWave<DK, NT, DELTA> m{a, lds, rows.first, rows.count, (rows.count + kChunk - 1) / kChunk,
                                   h / (a.v_heads / a.k_heads), h * a.v_dim + slab * 16 * NT, ws, step, w, lane, n, g};
  // all pass the same barriers: one before the chunks and three (two without beta) in each
  if (wave < 4) {
    __builtin_amdgcn_s_setprio(3);  // the chain first: the others have time
    float* st = a.state + ((slot * a.v_heads + h) * DK + w * (DK / 4) + 4 * g * (DK / 64)) * (int64_t)a.v_dim +
                slab * 16 * NT + n;
    carry_state<DK, NT, DELTA>(m, st, a.has_state && a.has_state[b] != 0);
  } else if (wave < 8) {
    write_outputs<DK, NT, DELTA>(m);
  } else {
    feed_chain<DK, NT, DELTA>(m);
  }
}

// ---- whole heads ------------------------------------------------------------------
// Where there are sequences and heads enough, a workgroup of eight waves carries 128
// columns, a wave 16 of them over all rows of the state: every product then leaves its
// rows where the next product's right operand wants them, and nothing passes between
// waves but what all of them read, the chunk's left operands in LDS.
template <int DK, bool DELTA>
struct HeadLds {
  static constexpr int kRow = DK * 2 + 16, kValueRow = 128 * 2 + 16;
  static constexpr int kSlot = 0, kSlotBytes = DELTA ? Slot::kBytesDelta : Slot::kBytesLinear;
  static constexpr int kTurned = kSlot + kSlotBytes;             // K^T: [step][tile of the state's rows]
  static constexpr int kQueries = kTurned + DK / 16 * 2 * 1024;
  static constexpr int kKeys = kQueries + kChunk * kRow;
  static constexpr int kValues = kKeys + kChunk * kRow;          // then the results
  static constexpr int kBytes = kValues + kChunk * kValueRow;
};

template <int DK, bool DELTA>
__global__ __launch_bounds__(512, 2) void gdn_head_kernel(GdnArgs a) {
  using L = HeadLds<DK, DELTA>;
  constexpr int TW = DK / 64, KS = DK / 32, P = DELTA ? 3 : 2;
  constexpr int kPieces = DK / 8, kLoads = DK / 64;              // of a key row; of a thread
  constexpr int kSlotPieces = L::kSlotBytes / 16, kSlotLoads = (kSlotPieces + 511) / 512;
  __shared__ __align__(16) uint8_t lds[L::kBytes];
  const int slabs = a.v_dim / 128;
  const int64_t turn = blockIdx.x / 8, pair = (turn / slabs) * 8 + blockIdx.x % 8;
  const int slab = (int)(turn % slabs);
  if (pair >= a.B * a.v_heads) return;
  const int b = by_length(a, (int)(pair / a.v_heads)), h = (int)(pair % a.v_heads), hk = h / (a.v_heads / a.k_heads);
  const int64_t index = a.index ? __builtin_amdgcn_readfirstlane(a.index[b]) : b;
  if (index < 0 || index >= a.num_states) return;
  const int t = threadIdx.x, lane = t % 64, n = lane % 16, g = lane / 16;
  const int w = __builtin_amdgcn_readfirstlane(t / 64);
  const Rows rows = rows_of(a, b);
  if (is_long(a, rows.count)) return;
  const int chunks = (rows.count + kChunk - 1) / kChunk;
  const int64_t col = (int64_t)h * a.v_dim + slab * 128;
  const int64_t ws_step = (int64_t)a.v_heads * L::kSlotBytes;
  const uint8_t* ws = static_cast<const uint8_t*>(a.workspace) + (rows.first / kChunk + b) * ws_step +
                      (int64_t)h * L::kSlotBytes;

  // tile q TW + i, register r: state row q DK / 4 + (4 g + r) TW + i
  float* st = a.state + (index * a.v_heads + h) * DK * (int64_t)a.v_dim + slab * 128 + 16 * w + n;
  auto state_at = [&](int x, int r) { return st + (int64_t)(x / TW * (DK / 4) + (4 * g + r) * TW + x % TW) * a.v_dim; };
  float4_t S[DK / 16];
  const bool load = a.has_state && a.has_state[b] != 0;
#pragma unroll
  for (int x = 0; x < DK / 16; ++x)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[x][r] = load ? *state_at(x, r) : 0.0f;

  struct {
    u32x4_t k[kLoads], q[kLoads], v[2], s[kSlotLoads];
  } next;
  auto fetch = [&](int ch) {
    const int64_t row0 = rows.first + (int64_t)ch * kChunk;
    const int last = min(kChunk, rows.count - ch * kChunk) - 1;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t r = row0 + min((i * 512 + t) / kPieces, last);
      const int at = hk * DK + t % kPieces * 8;
      next.k[i] = *reinterpret_cast<const u32x4_t*>(a.k + r * a.ldk + at);
      next.q[i] = *reinterpret_cast<const u32x4_t*>(a.q + r * a.ldq + at);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      next.v[i] = *reinterpret_cast<const u32x4_t*>(a.v + (row0 + min(i * 32 + t / 16, last)) * a.ldv + col + t % 16 * 8);
#pragma unroll
    for (int i = 0; i < kSlotLoads; ++i)
      next.s[i] = *reinterpret_cast<const u32x4_t*>(ws + ch * ws_step + min(i * 512 + t, kSlotPieces - 1) * 16);
  };
  auto put = [&] {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = (i * 512 + t) / kPieces * L::kRow + t % kPieces * 16;
      *reinterpret_cast<u32x4_t*>(lds + L::kKeys + at) = next.k[i];
      *reinterpret_cast<u32x4_t*>(lds + L::kQueries + at) = next.q[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<u32x4_t*>(lds + L::kValues + (i * 32 + t / 16) * L::kValueRow + t % 16 * 16) = next.v[i];
#pragma unroll
    for (int i = 0; i < kSlotLoads; ++i)
      if (i * 512 + t < kSlotPieces) *reinterpret_cast<u32x4_t*>(lds + L::kSlot + (i * 512 + t) * 16) = next.s[i];
  };
  // K^T, a quarter of its rows and a step of 32 tokens a wave, transposed within the lane
  auto turn_keys = [&] {
    const int q = w % 4, s = w / 4;
    uint32_t z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* from = lds + L::kKeys + (32 * s + (j / 4) * 16 + 4 * g + j % 4) * L::kRow + (q * (DK / 4) + n * TW) * 2;
      if constexpr (TW == 2)
        z[j] = *reinterpret_cast<const uint32_t*>(from);
      else
        z[j] = *reinterpret_cast<const uint16_t*>(from);
    }
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = i ? high_halves(z[2 * j], z[2 * j + 1]) : low_halves(z[2 * j], z[2 * j + 1]);
      *reinterpret_cast<uint4*>(lds + L::kTurned + (s * (DK / 16) + q * TW + i) * 1024 + lane * 16) =
          make_uint4(e[0], e[1], e[2], e[3]);
    }
  };
  // step s of row tile i of the keys or queries, in the order of the state's planes
  auto rows_at = [&](int area, int i, int s) {
    const uint8_t* row = lds + area + (16 * i + n) * L::kRow + 64 * s;
    if constexpr (TW == 2) return *reinterpret_cast<const uint4*>(row + 16 * g);
    const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * g), y = *reinterpret_cast<const uint2*>(row + 32 + 8 * g);
    return make_uint4(x.x, x.y, y.x, y.y);
  };
  auto block = [&](int at, int p, int i, int s) {
    return *reinterpret_cast<const uint4*>(lds + L::kSlot + at + (p * kBlocks + block_of(i, s)) * kBlockBytes + lane * 16);
  };
  auto decays = [&](int at, int i) { return *reinterpret_cast<const float4_t*>(lds + L::kSlot + at + (16 * i + 4 * g) * 4); };
  // rows of tiles 2 s and 2 s + 1 as planes of a right operand
  auto planes_of = [&](const float4_t& x, const float4_t& y, auto& out) {
    constexpr int N = sizeof(out) / sizeof(out[0]);
    uint32_t z[4][N];
    split_pair(x[0], x[1], z[0]);
    split_pair(x[2], x[3], z[1]);
    split_pair(y[0], y[1], z[2]);
    split_pair(y[2], y[3], z[3]);
#pragma unroll
    for (int p = 0; p < N; ++p) out[p] = make_uint4(z[0][p], z[1][p], z[2][p], z[3][p]);
  };

  if (chunks > 0) fetch(0);
  for (int ch = 0; ch < chunks; ++ch) {
    put();
    __syncthreads();
    turn_keys();
    if (ch + 1 < chunks) fetch(ch + 1);
    float4_t o[4], N[4];
    {
      uint4 z[KS][P];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (TW == 2) {
          const float4_t x = {S[2 * s][0], S[2 * s + 1][0], S[2 * s][1], S[2 * s + 1][1]};
          const float4_t y = {S[2 * s][2], S[2 * s + 1][2], S[2 * s][3], S[2 * s + 1][3]};
          planes_of(x, y, z[s]);
        } else {
          planes_of(S[2 * s], S[2 * s + 1], z[s]);
        }
      }
      float4_t ks[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = ks[i] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 x[4];
        if (DELTA) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = rows_at(L::kKeys, i, s);
#pragma unroll
          for (int p = P - 1; p >= 0; --p)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[i] = mfma_bf16(x[i], z[s][p], ks[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = rows_at(L::kQueries, i, s);
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mfma_bf16(x[i], z[s][p], o[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4_t decay = decays(Slot::kDecay, i);
        o[i] *= decay * a.scale;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          N[i][r] = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(
                        lds + L::kValues + (16 * i + 4 * g + r) * L::kValueRow + (16 * w + n) * 2) << 16);
        if (DELTA) N[i] -= decay * ks[i];
      }
    }
    if (DELTA) {  // N = T R
      uint4 r[2][3];
      planes_of(N[0], N[1], r[0]);
      planes_of(N[2], N[3], r[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4_t acc[3] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int s = 0; s <= i / 2; ++s) {
          const uint4 t0 = block(Slot::kT, 0, i, s), t1 = block(Slot::kT, 1, i, s), t2 = block(Slot::kT, 2, i, s);
          acc[0] = mfma_bf16(t0, r[s][0], acc[0]);
          acc[1] = mfma_bf16(t1, r[s][0], acc[1]);
          acc[2] = mfma_bf16(t2, r[s][0], acc[2]);
          acc[1] = mfma_bf16(t0, r[s][1], acc[1]);
          acc[2] = mfma_bf16(t1, r[s][1], acc[2]);
          acc[2] = mfma_bf16(t0, r[s][2], acc[2]);
        }
        N[i] = (acc[2] + acc[1]) + acc[0];
      }
    }
    {
      constexpr int PN = DELTA ? 2 : 1;  // without beta N is V, one plane
      uint4 x[2][PN];
      planes_of(N[0], N[1], x[0]);
      planes_of(N[2], N[3], x[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s <= i / 2; ++s) {
          const uint4 p0 = block(Slot::kP, 0, i, s);
          o[i] = mfma_bf16(block(Slot::kP, 1, i, s), x[s][0], o[i]);
          if constexpr (DELTA) o[i] = mfma_bf16(p0, x[s][1], o[i]);
          o[i] = mfma_bf16(p0, x[s][0], o[i]);
        }
    }
    wave_lds_fence();  // the results go where this wave's values were
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<uint16_t*>(lds + L::kValues + (16 * i + 4 * g + r) * L::kValueRow + (16 * w + n) * 2) =
            __builtin_bit_cast(uint16_t, (__bf16)o[i][r]);
    uint4 u[2][3];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      planes_of(N[2 * s] * decays(Slot::kLeft, 2 * s), N[2 * s + 1] * decays(Slot::kLeft, 2 * s + 1), u[s]);
    const float whole = reinterpret_cast<const float*>(lds + L::kSlot + Slot::kDecay)[63];
    __syncthreads();
    // S' = e^G S + K^T (e^(G_64 - G) N)
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) S[x] *= whole;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 k[DK / 16];
#pragma unroll
      for (int x = 0; x < DK / 16; ++x)
        k[x] = *reinterpret_cast<const uint4*>(lds + L::kTurned + (s * (DK / 16) + x) * 1024 + lane * 16);
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int x = 0; x < DK / 16; ++x) S[x] = mfma_bf16(k[x], u[s][p], S[x]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 32 + t / 16;
      if (r < rows.count - ch * kChunk)
        *reinterpret_cast<u32x4_t*>(a.out + (rows.first + (int64_t)ch * kChunk + r) * a.ldo + col + t % 16 * 8) =
            *reinterpret_cast<const u32x4_t*>(lds + L::kValues + r * L::kValueRow + t % 16 * 16);
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < DK / 16; ++x)
#pragma unroll
    for (int r = 0; r < 4; ++r) *state_at(x, r) = S[x][r];
}

size_t gdn_prefill_workspace(int64_t T, int64_t B, int, int v_heads, int, int) {
  return T == 0 ? 0 : (size_t)chunk_slots(T, B) * v_heads * Slot::kBytesDelta;
}

template <int DK, bool DELTA>
static hipError_t launch_prefill(const GdnArgs& a, hipStream_t stream) {
  if (a.T > 0) {
    const int64_t slots = (chunk_slots(a.T, a.B) + 7) / 8 * 8;
    const dim3 grid((unsigned)(slots * (a.v_heads / a.k_heads)), a.k_heads);
    gdn_chunk_kernel<DK, DELTA><<<grid, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t pairs = (a.B * a.v_heads + 7) / 8 * 8;
  // Whole heads where they fill the GPU, a workgroup on each CU: 5.6 us a chunk for 128
  // columns against four times 2.2 us for 32.  32 heads of 128: 24 prompts of up to 1000
  // tokens take 331 us (456 column by column), 12 of 100 55 us (70), 8 of 2048 319 us (426),
  // 24 of 1000 without beta 294 us (372); 6 of up to 8192, 192 heads, 893 us (699).  A
  // sequence that alone would outlast the rest goes column by column all the same -- only
  // the device knows which, and there can be no more than `most` -- in a launch of its own
  // before: one of 8192 beside eleven of 100 takes 379 us (349), without beta 237 (330).
  const int64_t heads = (int64_t)a.v_heads * (a.v_dim / 128);
  if (a.v_dim % 128 == 0 && a.B * heads >= kCUs) {
    const int64_t most = std::min(a.B, 2 * kCUs / (3 * heads));
    if (most > 0) {
      const int64_t some = (most * a.v_heads + 7) / 8 * 8;
      gdn_state_kernel<DK, 2, DELTA><<<(unsigned)(some * (a.v_dim / 32)), 768, 0, stream>>>(a, true);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    gdn_head_kernel<DK, DELTA><<<(unsigned)(pairs * (a.v_dim / 128)), 512, 0, stream>>>(a);
    return hipGetLastError();
  }
  // The launch runs in rounds.  With keys of 128 a workgroup fills a CU's LDS or its waves, so a
  // round is one for each CU; one of 32 columns takes about 1.4 times as long as one of 16, and
  // without beta one of 64 about 1.6 times as long as one of 32.  So 16 columns where they fit in
  // one round (32 heads of 128, 8192 tokens: 238 us against 334 with 32), else 32 (2 x 4096
  // tokens: 205 against 241 with 16; 3 x 4096: 365 against 390; 4 x 4096: 408 against 520), or 64
  // without beta where 32 would not fit in one (4 x 4096: 222 us against 268 with 32; 6 of up to
  // 8192: 428 against 467).  Where one sequence is far longer than the rest the smaller width can
  // be the faster (4096 and 1500 tokens: 163 us with 16 columns, 179 with 32), which the host
  // cannot know.  With keys of 64 two workgroups of 16 columns share a CU, so that up to two
  // rounds' worth of them would be as fast or faster (3 x 4096: 305 us against 331 with 32, 5 x
  // 300: 50 against 56; 2 x 4096: 187 against 180); the rule does not tell them apart.
  const bool one_round = pairs * (a.v_dim / 16) <= kCUs;
  const bool wide = !DELTA && a.v_dim % 64 == 0 && pairs * (a.v_dim / 32) > kCUs;
  const unsigned grid = (unsigned)(pairs * (a.v_dim / (wide ? 64 : (one_round ? 16 : 32))));
  if (one_round)
    gdn_state_kernel<DK, 1, DELTA><<<grid, 768, 0, stream>>>(a, false);
  else if (!wide)
    gdn_state_kernel<DK, 2, DELTA><<<grid, 768, 0, stream>>>(a, false);
  else if constexpr (!DELTA)
    gdn_state_kernel<DK, 4, DELTA><<<grid, 768, 0, stream>>>(a, false);
  return hipGetLastError();
}

hipError_t launch_gdn_prefill(const GdnArgs& a, hipStream_t stream) {
  if (a.k_dim == 64) return a.beta ? launch_prefill<64, true>(a, stream) : launch_prefill<64, false>(a, stream);
  return a.beta ? launch_prefill<128, true>(a, stream) : launch_prefill<128, false>(a, stream);
}

}  // namespace nvfp4

// One token of the gated delta rule for each of many sequences.
//
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// (without beta: u = v).  The columns of S do not touch each other, so a workgroup
// takes 32 or 128 of them, 256 threads holding 4 columns of a few rows each in
// registers.  Both column sums, S^T k and S^T q, are taken from the decayed state
// before its update, S'^T q = S^T q + (q . k) u, so that one reduction over the rows
// (lanes, then the four waves through LDS) serves both and the state is read once.
//
// Bound by HBM: the binary32 state in and out.  128 columns are whole rows, 64 KB in
// one piece (256 sequences of 32 heads of 128 x 128: 208 us against 222 with pieces of
// 128 bytes); fewer heads than CUs take 32, four workgroups to a head.  States beyond
// what the last-level cache keeps from one token to the next -- other layers' come in
// between -- are hinted as read once, and written so where they exceed it by themselves:
// 188 us, 5.7 TB/s (203 with loads hinted alone; 61 sequences: 43 us with loads, 45 with
// both, 49 with neither).
#include "common.hpp"
#include "mixers.hpp"
#include "mixers_device.hpp"

namespace nvfp4 {

typedef float floatx4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Adds each value up over the row groups of a wave (lanes STEP, 2 STEP, ... apart).
template <int STEP>
__device__ __forceinline__ float over_rows(float x) {
#pragma unroll
  for (int d = STEP; d < 64; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// COLS columns of one head's state: COLS / 4 lanes of 4 columns each side by side, the
// 1024 / COLS groups of them DK COLS / 1024 rows each.
// STREAM: 1: loads of the state are hinted as read once, 2: its stores too.
template <int DK, int COLS, bool DELTA, int STREAM>
__global__ __launch_bounds__(256) void gdn_step_kernel(GdnArgs a) {
  constexpr int kLanes = COLS / 4, R = DK * COLS / 1024;
  const int b = blockIdx.z, h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
  const int64_t slot = a.index ? a.index[b] : b;
  if (slot < 0 || slot >= a.num_states) return;
  const int c4 = threadIdx.x % kLanes, rg = threadIdx.x / kLanes, wave = threadIdx.x / 64;
  const int col = blockIdx.x * COLS + c4 * 4, row = rg * R;

  float* st = a.state + ((slot * a.v_heads + h) * DK + row) * a.v_dim + col;
  floatx4_t S[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const floatx4_t* from = reinterpret_cast<const floatx4_t*>(st + (int64_t)r * a.v_dim);
    S[r] = STREAM > 0 ? __builtin_nontemporal_load(from) : *from;
  }
  const float decay = expf(a.g[b * a.ldg + h]);
  const float beta = DELTA ? a.beta[b * a.ldb + h] : 1.0f;
  const uint2 vw = *reinterpret_cast<const uint2*>(a.v + b * a.ldv + (int64_t)h * a.v_dim + col);
  const uint16_t* kp = a.k + b * a.ldk + hk * DK + row;
  const uint16_t* qp = a.q + b * a.ldq + hk * DK + row;
  float k[R], q[R], qk = 0;
  floatx4_t ks = {0, 0, 0, 0}, qs = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < R; ++r) {
    k[r] = bf16_value(kp[r]), q[r] = bf16_value(qp[r]);
    S[r] *= decay;
    ks += S[r] * k[r];
    qs += S[r] * q[r];
    qk += q[r] * k[r];
  }
  __shared__ floatx4_t part[2][4][kLanes];  // [k sums, q sums][wave][column group]
  __shared__ float dots[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ks[e] = over_rows<kLanes>(ks[e]), qs[e] = over_rows<kLanes>(qs[e]);
  qk = over_rows<kLanes>(qk);
  if (threadIdx.x % 64 < kLanes) {
    part[0][wave][c4] = ks;
    part[1][wave][c4] = qs;
    if (c4 == 0) dots[wave] = qk;
  }
  __syncthreads();
  ks = (part[0][0][c4] + part[0][1][c4]) + (part[0][2][c4] + part[0][3][c4]);
  qs = (part[1][0][c4] + part[1][1][c4]) + (part[1][2][c4] + part[1][3][c4]);
  qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
  floatx4_t u = {bf16_value(vw.x & 0xFFFF), bf16_value(vw.x >> 16), bf16_value(vw.y & 0xFFFF), bf16_value(vw.y >> 16)};
  if (DELTA) u = beta * (u - ks);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    S[r] += k[r] * u;
    floatx4_t* to = reinterpret_cast<floatx4_t*>(st + (int64_t)r * a.v_dim);
    if (STREAM > 1)
      __builtin_nontemporal_store(S[r], to);
    else
      *to = S[r];
  }
  if (rg == 0) {
    const floatx4_t o = a.scale * (qs + qk * u);
    *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)h * a.v_dim + col) =
        make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
  }
}

template <int DK, int COLS, int STREAM>
static void launch_cols(const GdnArgs& a, hipStream_t stream) {
  const dim3 grid(a.v_dim / COLS, a.v_heads, (unsigned)a.B), block(256);
  if (a.beta)
    gdn_step_kernel<DK, COLS, true, STREAM><<<grid, block, 0, stream>>>(a);
  else
    gdn_step_kernel<DK, COLS, false, STREAM><<<grid, block, 0, stream>>>(a);
}

template <int DK>
static void launch_step(const GdnArgs& a, hipStream_t stream) {
  constexpr int64_t kCache = (int64_t)256 << 20;  // the last-level cache
  const int64_t bytes = a.B * a.v_heads * DK * a.v_dim * 4;
  if (a.v_dim % 128 != 0 || a.B * a.v_heads < 2 * kCUs)
    launch_cols<DK, 32, 0>(a, stream);
  else if (bytes >= kCache)
    launch_cols<DK, 128, 2>(a, stream);
  else if (bytes >= kCache / 4)
    launch_cols<DK, 128, 1>(a, stream);
  else
    launch_cols<DK, 128, 0>(a, stream);
}

hipError_t launch_gdn_step(const GdnArgs& a, hipStream_t stream) {
  a.k_dim == 64 ? launch_step<64>(a, stream) : launch_step<128>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4

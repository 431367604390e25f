// Gated linear attention with the delta rule (the Gated-DeltaNet recurrence), token
// by token, for single tokens and for prompts.
//
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// (without beta: u = v).  The columns of S do not touch each other, so a
// workgroup takes 32 of them: 256 threads hold 4 columns of k_dim / 32 rows each
// in registers.  Both column sums of a token, S^T k and S^T q, are taken from the
// decayed state before its update, S'^T q = S^T q + (q . k) u, so that one
// reduction over the rows (lanes, then the four waves through LDS) serves both.
// Bound by HBM for one token (the fp32 state is read and written once).
#include "common.hpp"
#include "mixers.hpp"

namespace nvfp4 {

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

constexpr int kCols = 32;  // state columns of a workgroup

template <int DK, bool DELTA, bool PREFILL>
__global__ __launch_bounds__(256) void gdn_recurrent_kernel(GdnArgs a) {
  constexpr int R = DK / 32;  // rows of a thread
  const int b = blockIdx.z, h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
  const int64_t slot = a.index ? a.index[b] : b;
  if (slot < 0 || slot >= a.num_states) return;
  const int c4 = threadIdx.x % 8, rg = threadIdx.x / 8, wave = threadIdx.x / 64;
  const int col = blockIdx.x * kCols + c4 * 4, row = rg * R;
  __shared__ float4 part[2][2][4][8];  // [token parity][k sums, q sums][wave][column group]
  __shared__ float dots[2][4];

  float* st = a.state + ((slot * a.v_heads + h) * DK + row) * a.v_dim + col;
  float4 S[R];
  const bool load = !PREFILL || (a.has_state && a.has_state[b] != 0);
#pragma unroll
  for (int r = 0; r < R; ++r)
    S[r] = load ? *reinterpret_cast<const float4*>(st + (int64_t)r * a.v_dim) : make_float4(0, 0, 0, 0);

  int64_t first = b, last = b + 1;
  if (PREFILL) {
    first = min(max((int64_t)a.cu[b], (int64_t)0), a.T);
    last = min(max((int64_t)a.cu[b + 1], first), a.T);
  }
  for (int64_t t = first; t < last; ++t) {
    const int par = (int)(t - first) & 1;
    const float decay = expf(a.g[t * a.ldg + h]);
    const uint16_t* kp = a.k + t * a.ldk + hk * DK + row;
    const uint16_t* qp = a.q + t * a.ldq + hk * DK + row;
    float k[R], q[R];
    float4 ks = make_float4(0, 0, 0, 0), qs = ks;
    float qk = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      k[r] = bf16_value(kp[r]), q[r] = bf16_value(qp[r]);
      S[r].x *= decay, S[r].y *= decay, S[r].z *= decay, S[r].w *= decay;
      ks.x += S[r].x * k[r], ks.y += S[r].y * k[r], ks.z += S[r].z * k[r], ks.w += S[r].w * k[r];
      qs.x += S[r].x * q[r], qs.y += S[r].y * q[r], qs.z += S[r].z * q[r], qs.w += S[r].w * q[r];
      qk += q[r] * k[r];
    }
#pragma unroll
    for (int d = 8; d < 64; d *= 2) {
      ks.x += __shfl_xor(ks.x, d), ks.y += __shfl_xor(ks.y, d), ks.z += __shfl_xor(ks.z, d), ks.w += __shfl_xor(ks.w, d);
      qs.x += __shfl_xor(qs.x, d), qs.y += __shfl_xor(qs.y, d), qs.z += __shfl_xor(qs.z, d), qs.w += __shfl_xor(qs.w, d);
      qk += __shfl_xor(qk, d);
    }
    if (threadIdx.x % 64 < 8) {
      part[par][0][wave][c4] = ks;
      part[par][1][wave][c4] = qs;
      if (c4 == 0) dots[par][wave] = qk;
    }
    __syncthreads();
    ks = part[par][0][0][c4], qs = part[par][1][0][c4], qk = dots[par][0];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 x = part[par][0][w][c4], y = part[par][1][w][c4];
      ks.x += x.x, ks.y += x.y, ks.z += x.z, ks.w += x.w;
      qs.x += y.x, qs.y += y.y, qs.z += y.z, qs.w += y.w;
      qk += dots[par][w];
    }
    const uint2 vw = *reinterpret_cast<const uint2*>(a.v + t * a.ldv + (int64_t)h * a.v_dim + col);
    float4 u = make_float4(bf16_value(vw.x & 0xFFFF), bf16_value(vw.x >> 16), bf16_value(vw.y & 0xFFFF),
                           bf16_value(vw.y >> 16));
    if (DELTA) {
      const float beta = a.beta[t * a.ldb + h];
      u = make_float4(beta * (u.x - ks.x), beta * (u.y - ks.y), beta * (u.z - ks.z), beta * (u.w - ks.w));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      S[r].x += k[r] * u.x, S[r].y += k[r] * u.y, S[r].z += k[r] * u.z, S[r].w += k[r] * u.w;
    }
    if (rg == 0) {
      const uint32_t lo = bf16_bits(a.scale * (qs.x + qk * u.x)) | ((uint32_t)bf16_bits(a.scale * (qs.y + qk * u.y)) << 16);
      const uint32_t hi = bf16_bits(a.scale * (qs.z + qk * u.z)) | ((uint32_t)bf16_bits(a.scale * (qs.w + qk * u.w)) << 16);
      *reinterpret_cast<uint2*>(a.out + t * a.ldo + (int64_t)h * a.v_dim + col) = make_uint2(lo, hi);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(st + (int64_t)r * a.v_dim) = S[r];
}

template <int DK, bool PREFILL>
static void launch_recurrent(const GdnArgs& a, hipStream_t stream) {
  const dim3 grid(a.v_dim / kCols, a.v_heads, (unsigned)a.B), block(256);
  if (a.beta)
    gdn_recurrent_kernel<DK, true, PREFILL><<<grid, block, 0, stream>>>(a);
  else
    gdn_recurrent_kernel<DK, false, PREFILL><<<grid, block, 0, stream>>>(a);
}

hipError_t launch_gdn_step(const GdnArgs& a, hipStream_t stream) {
  a.k_dim == 64 ? launch_recurrent<64, false>(a, stream) : launch_recurrent<128, false>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4

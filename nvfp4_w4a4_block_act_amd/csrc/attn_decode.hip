// Attention of one new token over the paged key-value cache.
//
// One pass over the cached tokens with the running maximum m and sum l of the
// softmax: a score s moves m to m' = max(m, s), and the sums taken so far are
// scaled by e^(m - m').  A workgroup takes one query head of one sequence; its
// four waves take every fourth token, a lane head_dim / 64 elements of the rows,
// and join through LDS at the end.
#include "common.hpp"
#include "mixers.hpp"

namespace nvfp4 {

constexpr float kNone = -3.402823466e38f;  // running maximum before any token: finite, so that differences are numbers

template <int DIM, bool FP8>
__global__ __launch_bounds__(256) void attn_decode_kernel(AttnArgs a) {
  constexpr int E = DIM / 64;
  const int h = blockIdx.x, b = blockIdx.y;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const nvfp4_kv_cache& c = a.cache;
  const int kvh = h / (a.q_heads / c.kv_heads);
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int begin = a.window ? max(0, len - a.window) : 0;
  const float kg = FP8 ? *c.k_amax / 448.0f : 1.0f, vg = FP8 ? *c.v_amax / 448.0f : 1.0f;

  float q[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e)
    q[e] = __uint_as_float((uint32_t)a.q[(int64_t)b * a.ldq + h * DIM + lane * E + e] << 16);
  float m = kNone, l = 0;
  for (int t = begin + wave; t < len; t += 4) {
    const int page = a.table[(int64_t)b * a.ldt + t / c.page_size];
    if (page < 0 || page >= c.num_pages) continue;
    const int64_t at = page * c.page_stride + (int64_t)(t % c.page_size) * c.token_stride + (int64_t)kvh * c.head_stride +
                       lane * E;
    float k[E], v[E], s = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (FP8) {
        k[e] = __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(c.k)[at + e], 0);
        v[e] = __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(c.v)[at + e], 0);
      } else {
        k[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(c.k)[at + e] << 16);
        v[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(c.v)[at + e] << 16);
      }
      s += q[e] * k[e];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    s *= a.scale * kg;
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + p * v[e];
  }
  __shared__ float ms[4], ls[4], os[4][DIM];
#pragma unroll
  for (int e = 0; e < E; ++e) os[wave][lane * E + e] = o[e];
  if (lane == 0) ms[wave] = m, ls[wave] = l;
  __syncthreads();
  if (threadIdx.x < DIM) {
    float top = kNone, sum = 0, out = 0;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ms[w]);
    for (int w = 0; w < 4; ++w) {
      const float f = ls[w] > 0 ? expf(ms[w] - top) : 0.0f;
      sum += ls[w] * f;
      out += os[w][threadIdx.x] * f;
    }
    const float r = sum > 0 ? out / sum * vg : 0.0f;
    a.out[(int64_t)b * a.ldo + h * DIM + threadIdx.x] = __builtin_bit_cast(uint16_t, (__bf16)r);
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)b * a.q_heads + h] = sum > 0 ? top + logf(sum) : -INFINITY;
  }
}

size_t attn_decode_workspace(int64_t, int, int, int, int64_t, int64_t) { return 0; }

template <int DIM>
static void launch_dim(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid(a.q_heads, (unsigned)a.B), block(256);
  if (a.cache.dtype == NVFP4_E4M3)
    attn_decode_kernel<DIM, true><<<grid, block, 0, stream>>>(a);
  else
    attn_decode_kernel<DIM, false><<<grid, block, 0, stream>>>(a);
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream) {
  if (a.cache.head_dim == 64)
    launch_dim<64>(a, stream);
  else if (a.cache.head_dim == 128)
    launch_dim<128>(a, stream);
  else
    launch_dim<256>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4

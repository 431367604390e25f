// Append to the paged key-value cache, with the rotation by position.
//
// Every head of a token is a whole number of items of 16 elements, each two runs
// of 8: the two halves of 8 rotated pairs (runs rot / 2 apart, or next to each
// other where pairs are interleaved), or 16 elements that are not rotated.  Both
// layouts of the pairs take the same 8 table columns for an item.  A thread does
// one item: 16-byte loads, x1' = fl(fl(x1 c) - fl(x2 s)), x2' = fl(fl(x2 c) +
// fl(x1 s)) (contraction is off, so results are bit-exact), a rounding to bf16
// (the cache codec's input type, and what the attention reads), and for an E4M3
// cache the codec's own steps.  A workgroup takes one token, a thread for each item
// (up to 512), so that no wave runs a second, partly empty trip.  Bound by HBM: the
// rows in, the rows out and one table row for each token; a token's heads find the table
// row in the caches.  32768 tokens of 40 + 2 x 8 heads of 128, fp32 to FP8: 221 us,
// 6.1 TB/s (245 us with 256 threads a token; hinted loads 254, stores too 242).
#include <algorithm>

#include "common.hpp"
#include "kv_codec.hpp"
#include "mixers.hpp"
#include "mixers_device.hpp"

namespace nvfp4 {

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if (F32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint4 bf16_run(const float (&x)[8]) {
  return make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}

__device__ __forceinline__ uint2 coded_run(uint4 w, float g) {
  return make_uint2(kv_encode_pair(w.x, g) | (kv_encode_pair(w.y, g) << 16),
                    kv_encode_pair(w.z, g) | (kv_encode_pair(w.w, g) << 16));
}

template <bool F32, bool FP8>
__global__ __launch_bounds__(512) void kv_append_kernel(AppendArgs a) {
  const int64_t t = blockIdx.x;
  const nvfp4_kv_cache& c = a.cache;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= c.num_pages * c.page_size) return;
  const float* row = nullptr;
  if (a.rot > 0) {
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.max_pos) return;
    row = a.rope + pos * a.rot;
  }
  const int64_t base = (slot / c.page_size) * c.page_stride + (slot % c.page_size) * c.token_stride;
  const int per = c.head_dim / 16, half = a.rot / 2;
  const int nq = a.q ? a.q_heads * per : 0, nk = c.kv_heads * per;
  for (int item = threadIdx.x; item < nq + 2 * nk; item += blockDim.x) {
    const bool is_q = item < nq, is_v = item >= nq + nk;
    const int i = is_q ? item : (is_v ? item - nq - nk : item - nq);
    const int head = i / per, r = i % per;
    const bool turned = !is_v && r * 16 < a.rot;
    const int o1 = turned && !a.interleaved ? r * 8 : r * 16;
    const int o2 = turned && !a.interleaved ? half + r * 8 : r * 16 + 8;
    const void* src = is_q ? a.q : (is_v ? a.v : a.k);
    const int64_t from = t * (is_q ? a.ldq : (is_v ? a.ldv : a.ldk)) + (int64_t)head * c.head_dim;
    float x[8], y[8];
    load8<F32>(src, from + o1, x);
    load8<F32>(src, from + o2, y);
    if (turned) {
      float cs[8], sn[8];
      load8<true>(row, r * 8, cs);
      load8<true>(row, half + r * 8, sn);
      if (a.interleaved) {
        float z[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = x[j], z[j + 8] = y[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = z[2 * j], w = z[2 * j + 1];
          z[2 * j] = u * cs[j] - w * sn[j];
          z[2 * j + 1] = w * cs[j] + u * sn[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = z[j], y[j] = z[j + 8];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = x[j], w = y[j];
          x[j] = u * cs[j] - w * sn[j];
          y[j] = w * cs[j] + u * sn[j];
        }
      }
    }
    const uint4 b1 = bf16_run(x), b2 = bf16_run(y);
    if (is_q) {
      uint16_t* to = a.q_out + t * a.ldqo + (int64_t)head * c.head_dim;
      *reinterpret_cast<uint4*>(to + o1) = b1;
      *reinterpret_cast<uint4*>(to + o2) = b2;
    } else if (FP8) {
      const float g = kv_g_enc(is_v ? *c.v_amax : *c.k_amax);
      uint8_t* to = static_cast<uint8_t*>(is_v ? c.v : c.k) + base + (int64_t)head * c.head_stride;
      *reinterpret_cast<uint2*>(to + o1) = coded_run(b1, g);
      *reinterpret_cast<uint2*>(to + o2) = coded_run(b2, g);
    } else {
      uint16_t* to = static_cast<uint16_t*>(is_v ? c.v : c.k) + base + (int64_t)head * c.head_stride;
      *reinterpret_cast<uint4*>(to + o1) = b1;
      *reinterpret_cast<uint4*>(to + o2) = b2;
    }
  }
}

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream) {
  const int64_t items = (int64_t)((a.q ? a.q_heads : 0) + 2 * a.cache.kv_heads) * (a.cache.head_dim / 16);
  const dim3 grid((unsigned)a.T), block((unsigned)std::min<int64_t>(512, (items + 63) / 64 * 64));
  const bool fp8 = a.cache.dtype == NVFP4_E4M3;
  if (a.src_f32 && fp8)
    kv_append_kernel<true, true><<<grid, block, 0, stream>>>(a);
  else if (a.src_f32)
    kv_append_kernel<true, false><<<grid, block, 0, stream>>>(a);
  else if (fp8)
    kv_append_kernel<false, true><<<grid, block, 0, stream>>>(a);
  else
    kv_append_kernel<false, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4

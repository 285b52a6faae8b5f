// Attention over the paged cache, one warp per new token and query head.
//
//   z_j = f(scale * q . k_j) + slope * (j - p),  f(s) = cap tanh(s / cap)
//   over the visible keys j: j < len, j <= p or j < prefix, j > p - window;
//   out = sum_j e^z_j v_j / (sum_j e^z_j + e^sink),  lse = log of the divisor
//
// with the running maximum and sum of the softmax, 32-bit throughout.
#include <cuda_fp8.h>

#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128)
    paged_attention_kernel(const PagedKv kv, const PagedAttnArgs a, int32_t* err) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t t = item / a.heads;
  const int h = int(item - t * a.heads);
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  if (t >= a.tokens) return;
  const int b = a.starts ? paged_seq_of(a.starts, kv.batch, t, lane) : int(t);
  int32_t* e1 = lane == 0 ? err : nullptr;
  const int64_t len = paged_len(kv, b, e1);
  int64_t p = len - 1;
  if (a.starts) {
    const int64_t s0 = __ldcg(a.starts + b), s1 = __ldcg(a.starts + b + 1);
    if (t < s0 || t >= s1) return;
    p = len - (s1 - t);
  }
  const int64_t pre = a.prefix ? __ldcg(a.prefix + b) : 0;
  int64_t hi = p + 1 > pre ? p + 1 : pre;
  if (hi > len) hi = len;
  if (p < 0) hi = 0;
  const int64_t lo = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
  const int j = h / (a.heads / kv.kv_heads);
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = bf16_bits_to_f32(__ldcg(a.q + t * a.q_stride + int64_t(h) * D + lane * E + i));
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const float slope = a.slopes ? __ldcg(a.slopes + h) : 0.f;
  for (int64_t x = lo; x < hi; ++x) {
    const int page = paged_page(kv, b, x, e1);
    if (page < 0) continue;
    const int64_t row = paged_row(kv, page, j, x);
    float k[E], v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int64_t at = row * D + lane * E + i;
      if constexpr (FP8) {
        k[i] = e4m3_f32(static_cast<const uint8_t*>(kv.k)[at]);
        v[i] = e4m3_f32(static_cast<const uint8_t*>(kv.v)[at]);
      } else {
        k[i] = bf16_bits_to_f32(static_cast<const uint16_t*>(kv.k)[at]);
        v[i] = bf16_bits_to_f32(static_cast<const uint16_t*>(kv.v)[at]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
    s = warp_sum(s) * a.scale;
    if constexpr (FP8) s *= kv.k_scales[row];
    if (a.softcap > 0.f) s = cap_score(s, a.softcap, 1.f / a.softcap);
    s += slope * float(x - p);
    const float mn = fmaxf(m, s);
    const float al = mn == -INFINITY ? 1.f : expf(m - mn);
    const float w = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * al + w;
    const float wv = FP8 ? w * kv.v_scales[row] : w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * al + wv * v[i];
  }
  if (a.sinks) {
    const float s = __ldcg(a.sinks + h);
    const float mn = fmaxf(m, s);
    const float al = m == -INFINITY ? 0.f : expf(m - mn);
    m = mn;
    l = l * al + expf(s - mn);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= al;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const __nv_bfloat16 r = __float2bfloat16_rn(o[i] * inv);
    a.out[(t * a.heads + h) * D + lane * E + i] = *reinterpret_cast<const uint16_t*>(&r);
  }
  if (a.lse && lane == 0) a.lse[t * a.heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

cudaError_t launch(const PagedKv& kv, int D, bool fp8, const PagedAttnArgs& a, cudaStream_t s,
                   bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.tokens * a.heads + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (D == 64)
    return fp8 ? cudaLaunchKernelEx(&cfg, paged_attention_kernel<64, true>, kv, a, di->error_word)
               : cudaLaunchKernelEx(&cfg, paged_attention_kernel<64, false>, kv, a,
                                    di->error_word);
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_attention_kernel<128, true>, kv, a, di->error_word)
             : cudaLaunchKernelEx(&cfg, paged_attention_kernel<128, false>, kv, a,
                                  di->error_word);
}

}  // namespace

size_t paged_prefill_workspace_bytes(int) { return 16; }
cudaError_t launch_paged_prefill(const PagedKv& kv, int head_dim, bool fp8,
                                 const PagedAttnArgs& a, cudaStream_t s, bool pdl) {
  return launch(kv, head_dim, fp8, a, s, pdl);
}

}  // namespace tt

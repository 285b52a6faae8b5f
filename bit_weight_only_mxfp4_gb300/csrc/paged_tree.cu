// Attention of a tree of drafted tokens over the paged cache.
//
//   z = f(scale * q . k) + slope (place of the key - place of the token)
//   out = sum e^z v / (sum e^z + e^sink)
//
// over the cached tokens and those new ones that the token's mask row names.
#include "launch.h"
#include <cuda_fp8.h>

#include "paged.cuh"

namespace tt {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kWarps = 4;

// A CTA per (token, head); its warps take the keys in turn.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * kWarps)
    paged_tree_kernel(const PagedKv kv, const TreeArgs t, int32_t* err) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const PagedAttnArgs& a = t.attn;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int64_t tok = blockIdx.x / a.heads;
  const int h = int(blockIdx.x % a.heads), j = h / (a.heads / kv.kv_heads);
  auto start_of = [&](int b) {
    const int64_t s = __ldcg(a.starts + b);
    return s < 0 ? 0 : s > a.tokens ? a.tokens : s;
  };
  int b = -1;
  int64_t s0 = 0, s1 = 0;
  for (int c = 0; c < kv.batch && b < 0; ++c) {
    s0 = start_of(c);
    s1 = start_of(c + 1);
    if (tok >= s0 && tok < s1) b = c;
  }
  if (b < 0) return;
  const int n = int(s1 - s0), i = int(tok - s0);
  const int len = paged_len(kv, b, blockIdx.x == 0 ? err : nullptr), past = len - n;
  const int most = n < 32 * t.words ? n : 32 * t.words;
  auto sees = [&](int row, int k) {
    return k < most && (__ldcg(t.masks + (s0 + row) * t.words + (k >> 5)) >> (k & 31) & 1u);
  };
  auto depth_of = [&](int row) {
    int d = 0;
    for (int k = 0; k < most; ++k) d += sees(row, k);
    return d > 0 ? d - 1 : 0;
  };
  const int depth = depth_of(i);
  float q[E], o[E];
  float m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_bits_to_f32(__ldcg(a.q + tok * a.q_stride + int64_t(h) * D + lane * E + e));
    o[e] = 0.f;
  }
  const float slope = a.slopes ? __ldcg(a.slopes + h) : 0.f;
  for (int64_t p = warp; past + i >= 0 && p < len; p += kWarps) {
    const int k = int(p) - past;
    if (k >= 0 && !sees(i, k)) continue;
    const int far = (k < 0 ? int(p) : past + depth_of(k)) - past - depth;
    if (a.window > 0 && -far >= a.window) continue;
    const int page = paged_page(kv, b, p, err);
    if (page < 0) continue;
    const int64_t row = paged_row(kv, page, j, p);
    float kx[E], vx[E], dot = 0.f;
    for (int e = 0; e < E; ++e) {
      if constexpr (FP8) {
        auto value = [](const void* base, int64_t at, float s) {
          __half_raw r = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[at], __NV_E4M3);
          return __half2float(__half(r)) * s;
        };
        kx[e] = value(kv.k, row * D + lane * E + e, kv.k_scales[row]);
        vx[e] = value(kv.v, row * D + lane * E + e, kv.v_scales[row]);
      } else {
        kx[e] = bf16_bits_to_f32(static_cast<const uint16_t*>(kv.k)[row * D + lane * E + e]);
        vx[e] = bf16_bits_to_f32(static_cast<const uint16_t*>(kv.v)[row * D + lane * E + e]);
      }
      dot = fmaf(q[e], kx[e], dot);
    }
    float z = warp_sum(dot) * a.scale;
    if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
    z = (z + slope * float(far)) * kLog2e;
    const float m2 = fmaxf(m, z), f = m2 == -INFINITY ? 0.f : ex2(m - m2),
                w = m2 == -INFINITY ? 0.f : ex2(z - m2);
    m = m2;
    l = l * f + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * vx[e];
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (warp > 0) return;
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
  float sum[E] = {};
  for (int w = 0; w < kWarps; ++w) {
    const float f = mm == -INFINITY ? 0.f : ex2(s_m[w] - mm);
    ll += s_l[w] * f;
    for (int e = 0; e < E; ++e) sum[e] += s_o[w][lane * E + e] * f;
  }
  const int64_t row = tok * a.heads + h;
  const float inv = close_row(mm, ll, a.sinks, h, lane == 0 ? a.lse : nullptr, row);
  for (int e = 0; e < E; ++e) {
    const __nv_bfloat16 y = __float2bfloat16_rn(sum[e] * inv);
    a.out[row * D + lane * E + e] = *reinterpret_cast<const uint16_t*>(&y);
  }
}

}  // namespace

size_t paged_tree_workspace_bytes(int head_dim) { return 0; }

cudaError_t launch_paged_tree(const PagedKv& kv, int head_dim, bool fp8, const TreeArgs& a,
                              cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  auto kern = head_dim == 64 ? (fp8 ? paged_tree_kernel<64, true> : paged_tree_kernel<64, false>)
                             : (fp8 ? paged_tree_kernel<128, true> : paged_tree_kernel<128, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.attn.tokens * a.attn.heads));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, kv, a, di->error_word);
}

}  // namespace tt

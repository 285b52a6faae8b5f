// Log probabilities of given tokens, with entropy and top alternatives.
//
//   x = scale * logit;  lse = m + log sum e^(x - m)
//   logp = x[target] - lse;  H = log sum e^(x - m) - sum (x - m) e^(x - m) / sum e^(x - m)
#include "launch.h"
#include "common.cuh"

namespace tt {
namespace {

constexpr int kThreads = 256;
constexpr int kErrShape = 2;

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(__ldcg(static_cast<const uint16_t*>(row) + i));
  return __ldcg(static_cast<const float*>(row) + i);
}

// Larger for a larger logit, and of equal ones for the smaller index; never 0.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) {
  uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  if (x != x) u = 0x7fffffffu;
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return uint64_t(u) << 32 | (0xffffffffu - i);
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F f, T* part) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, part[w]);
  __syncthreads();
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a, int32_t* err) {
  __shared__ float fpart[kThreads / 32];
  __shared__ uint64_t kpart[kThreads / 32];
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + r * a.stride * (BF16 ? 2 : 4);
  float m = -INFINITY;
  for (int64_t i = tid; i < a.vocab; i += kThreads) {
    const float x = logit<BF16>(row, i) * a.scale;
    m = x != x || m != m ? NAN : fmaxf(m, x);
  }
  m = block_reduce(m, [](float x, float y) { return x != x || y != y ? NAN : fmaxf(x, y); }, fpart);
  float s = 0.f, e = 0.f;
  for (int64_t i = tid; i < a.vocab; i += kThreads) {
    const float y = logit<BF16>(row, i) * a.scale - m, w = expf(y);
    s += w;
    e += w > 0.f ? y * w : 0.f;
  }
  s = block_reduce(s, [](float x, float y) { return x + y; }, fpart);
  e = block_reduce(e, [](float x, float y) { return x + y; }, fpart);
  const float bad = m - m;  // NaN unless m is finite
  const float ls = logf(s) + bad;
  if (tid == 0) {
    if (a.entropy) a.entropy[r] = ls - e / s;
    if (a.logp) {
      const int t = __ldcg(a.targets + r);
      if (t >= a.vocab) flag_error(err, kErrShape);
      a.logp[r] = t < 0 ? 0.f : t >= a.vocab ? NAN : logit<BF16>(row, t) * a.scale - m - ls;
    }
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    uint64_t best = 0;
    for (int64_t i = tid; i < a.vocab; i += kThreads) {
      const uint64_t key = key_of(logit<BF16>(row, i), uint32_t(i));
      if (key < last && key > best) best = key;
    }
    last = block_reduce(best, [](uint64_t x, uint64_t y) { return x > y ? x : y; }, kpart);
    if (tid == 0) {
      const int32_t id = int32_t(0xffffffffu - uint32_t(last));
      a.top_ids[r * a.top + k] = id;
      if (a.top_logp) a.top_logp[r * a.top + k] = logit<BF16>(row, id) * a.scale - m - ls;
    }
  }
}

}  // namespace

size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top) { return 0; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, bool bf16, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return bf16 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, a, di->error_word)
              : cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, a, di->error_word);
}

}  // namespace tt

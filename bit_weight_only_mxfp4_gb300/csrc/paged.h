// Host-visible types and launchers of the paged key-value cache operators.
// Arguments are already validated by the C-ABI layer in api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace tt {

// tt_paged_kv after validation, with the page size as a shift.
struct PagedKv {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  const int32_t* page_table;
  const int32_t* lens;
  int num_pages, page_shift, kv_heads, batch, pages_per_seq;
};

struct RopeArgs {
  const uint64_t* turns;  // nullptr: no rotation
  int rot;
  bool interleaved;
  const int32_t* positions;  // nullptr: the place in the cache
  int axes;
  const uint8_t* pair_axis;
};

struct PagedAttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* starts;  // nullptr: one new token per sequence
  int64_t tokens;
  int heads;
  float scale, softcap;
  int window;
  const float* slopes;
  const float* sinks;
  const int32_t* prefix;
  uint16_t* out;
  float* lse;
  void* ws;
};

// Whether a kernel whose warps trade registers (setmaxnreg) was compiled with
// the registers per thread that its shares add up to: with fewer, a warp
// would wait for registers that the CTA does not have.  Asked once a kernel.
template <typename Kern>
bool has_registers(Kern kern, int regs) {
  cudaFuncAttributes at;
  return cudaFuncGetAttributes(&at, kern) == cudaSuccess && at.numRegs >= regs;
}

constexpr int kPagedMaxBatch = 1024;
constexpr int kPagedMaxGroup = 16;  // query heads per kv head
constexpr float kCapSmall = 256.f;  // caps up to here are taken from the exponential alone

// paged_append.cu
cudaError_t launch_rope_turns(const double* inv_freq, int n, uint64_t* turns, cudaStream_t s);
cudaError_t launch_paged_append(const PagedKv& kv, int head_dim, bool fp8, const uint16_t* q,
                                const uint16_t* k, const uint16_t* v, int64_t q_stride,
                                int64_t kv_stride, int64_t tokens, const int32_t* starts,
                                int heads, const RopeArgs& rope, uint16_t* q_out, cudaStream_t s,
                                bool pdl);

// paged_decode.cu, paged_prefill.cu
size_t paged_decode_workspace_bytes(int group, int head_dim);
cudaError_t launch_paged_decode(const PagedKv& kv, int head_dim, bool fp8,
                                const PagedAttnArgs& a, cudaStream_t s, bool pdl);
size_t paged_prefill_workspace_bytes(int head_dim);
cudaError_t launch_paged_prefill(const PagedKv& kv, int head_dim, bool fp8,
                                 const PagedAttnArgs& a, cudaStream_t s, bool pdl);

}  // namespace tt

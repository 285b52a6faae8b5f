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

// The caches of several layers: one geometry, a pool each.
constexpr int kMaxLayers = 128;  // TT_PAGED_MAX_LAYERS
struct PagedPools {
  int layers;
  void* k[kMaxLayers];
  void* v[kMaxLayers];
  float* k_scales[kMaxLayers];
  float* v_scales[kMaxLayers];
};

struct TreeArgs {
  PagedAttnArgs attn;  // (prefix unused)
  const uint32_t* masks;
  int words;
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


// paged_tree.cu
size_t paged_tree_workspace_bytes(int head_dim);
cudaError_t launch_paged_tree(const PagedKv& kv, int head_dim, bool fp8, const TreeArgs& a,
                              cudaStream_t s, bool pdl);

// draft.cu
constexpr int kMaxMaskWords = 8;  // TT_TREE_MAX_WORDS
cudaError_t launch_draft_tree(const int32_t* parents, const int32_t* starts, const int32_t* lens,
                              int batch, int64_t tokens, int words, uint32_t* masks,
                              int32_t* positions, cudaStream_t s, bool pdl);
cudaError_t launch_draft_accept(const int32_t* parents, const int32_t* drafts,
                                const int32_t* chosen, const int32_t* starts, int batch,
                                int64_t tokens, int width, int32_t* path, int32_t* counts,
                                int32_t* next, cudaStream_t s, bool pdl);
cudaError_t launch_paged_keep(const PagedKv& kv, const PagedPools& pools, int head_dim, bool fp8,
                              const int32_t* starts, const int32_t* path, int width,
                              const int32_t* counts, int32_t* lens_out, cudaStream_t s, bool pdl);

// pages.cu
size_t paged_pages_workspace_bytes(int64_t num_pages, int64_t batch, int64_t pages_per_seq);
cudaError_t launch_paged_resize(const PagedKv& kv, const int32_t* want, const uint8_t* held,
                                int32_t* table_out, int32_t* lens_out, int32_t* left, void* ws,
                                cudaStream_t s, bool pdl);
cudaError_t launch_paged_fork(const PagedKv& kv, const PagedPools& pools, int head_dim, bool fp8,
                              const int32_t* from, const uint8_t* held, int32_t* table_out,
                              int32_t* lens_out, int32_t* left, void* ws, cudaStream_t s, bool pdl);
cudaError_t launch_paged_compact(const PagedKv& kv, const PagedPools& pools, int head_dim,
                                 bool fp8, const uint8_t* held, int32_t* table_out, int32_t* span,
                                 void* ws, cudaStream_t s, bool pdl);

}  // namespace tt

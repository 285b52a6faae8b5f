// The paged key-value cache as the kernels see it: the addressing that the
// append and the attention kernels share.
//
// Token t of sequence b is row t % page_size of page table[b][t / page_size];
// a page holds, for every kv head, page_size rows of head_dim elements:
//   row index  (page * kv_heads + j) * page_size + t % page_size
// so the rows of one head and page are contiguous.  A table entry that is
// negative is a hole: its tokens have no row (masked in attention, dropped by
// the append).  An entry >= num_pages is an error (TT_ERR_SHAPE in the device
// error word) and is treated as a hole: nothing outside the pool is touched.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace tt {

constexpr int kErrShape = 2;  // TT_ERR_SHAPE
constexpr float kLog2e = 1.4426950408889634f;

// The page that holds token t of sequence b, or -1; t is inside the table.
__device__ __forceinline__ int paged_page(const PagedKv& kv, int b, int64_t t, int32_t* err) {
  const int p = __ldcg(kv.page_table + int64_t(b) * kv.pages_per_seq + (t >> kv.page_shift));
  if (p >= kv.num_pages) flag_error(err, kErrShape);
  return p >= 0 && p < kv.num_pages ? p : -1;
}

// Length of sequence b, brought into what the table can address (a length
// outside it is an error: TT_ERR_SHAPE in the device error word).  Tokens of
// a sequence are counted in 32 bits (the host checks the table's extent).
__device__ __forceinline__ int paged_len(const PagedKv& kv, int b, int32_t* err) {
  const int most = kv.pages_per_seq << kv.page_shift;
  const int n = __ldcg(kv.lens + b);
  if (n < 0 || n > most) flag_error(err, kErrShape);
  return n < 0 ? 0 : n > most ? most : n;
}

// Row of (page, kv head j, token t) in k, v and their scales.
__device__ __forceinline__ int64_t paged_row(const PagedKv& kv, int page, int j, int64_t t) {
  return ((int64_t(page) * kv.kv_heads + j) << kv.page_shift) + (t & ((1 << kv.page_shift) - 1));
}

// The sequence of flat token t: the number of starts[1 .. batch - 1] that
// are <= t, counted by the whole warp (starts ascend; empty sequences share
// a start).  With the loads in flight together this is one round trip to L2
// where a binary search is log2(batch).
__device__ __forceinline__ int paged_seq_of(const int32_t* starts, int batch, int64_t t,
                                            int lane) {
  int n = 0;
  for (int i = 1 + lane; i < batch; i += 32) n += __ldcg(starts + i) <= t;
  return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The end of a row from its maximum m (log2 units) and its sum l of weights
// 2^(z - m): the sink, the logarithm; returns the factor of the sum of
// weights times values.  l = 0: the row sees no key, its sink is all there is,
// and the result 0.  A sink of -infinity adds nothing; one of +infinity has
// the whole weight.
__device__ __forceinline__ float close_row(float m, float l, const float* sinks, int h,
                                           float* lse, int64_t row) {
  float f = 1.f;
  if (sinks) {
    const float sink = __ldcg(sinks + h);
    if (l == 0.f) {
      if (lse) lse[row] = sink;
      return 0.f;
    }
    const float z = sink * kLog2e, m2 = fmaxf(m, z);
    f = m == -INFINITY ? 0.f : ex2(m - m2);
    // z - m2 is no number where both are infinite
    l = l * f + (z == -INFINITY ? 0.f : z == m2 ? 1.f : ex2(z - m2));
    m = m2;
  }
  if (lse) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  return f * (l > 0.f ? 1.f / l : l == 0.f ? 0.f : l);  // a NaN stays one
}

}  // namespace tt

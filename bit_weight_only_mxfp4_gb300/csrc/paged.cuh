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

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The cap: c tanh(s / c) of a score s, both in log2 units (times log2 e).  With
// x = s / c and y = 2 x log2 e, tanh x = 1 - 2 / (1 + 2^y); 2^y may be infinite,
// its reciprocal is then 0.  That is off by about c 2^-22 absolutely, which is
// what counts in the exponent, also where s is far below c.  Caps above
// kCapSmall (2^-14 there, against the 2^-8 and 2^-11 of weights rounded to bf16
// and f16) have kernels of their own: they take it from |y| = kCapSeries
// (|x| = 0.25) on only, and below it
//   s (1 - x^2 / 3 + 2 x^4 / 15 - 17 x^6 / 315 + 62 x^8 / 2835)
// whose next term is below 2^-26: off by a few 2^-24 of s, and by 2^-19 of it at
// most beyond.  Measured with a cap
// of 50 / 500: 8192 prompt tokens, 16 / 4 heads of 128, all of a prefix of 7411
// seen, 765 / 774 us; the FP8 decode batch of 64 122.6 / 141.  (Both forms in one
// kernel: 890 / 915 and 126 / 144, and that batch without a cap 116 for 113.)
constexpr float kCapSeries = 0.72f;
constexpr float kFiniteMax = 3.4028234663852886e38f;
struct Cap {
  float top, per;  // c log2 e; y of s
};
__device__ __forceinline__ Cap cap_of(float c) {
  // finite, so that 0 * per is 0 with the smallest caps
  return {fminf(c * kLog2e, kFiniteMax), fminf(2.f / c, kFiniteMax)};
}
__device__ __forceinline__ float cap_small(float y, const Cap& c) {
  return fmaf(-2.f * c.top, rcp(1.f + ex2(y)), c.top);
}
constexpr float kCap1 = -1.f / 3.f, kCap2 = 2.f / 15.f, kCap3 = -17.f / 315.f, kCap4 = 62.f / 2835.f;
constexpr float kHalfLn2 = 0.34657359027997264f;  // x = y ln 2 / 2
__device__ __forceinline__ float cap_series(float s, const Cap& c) {
  const float x = s * c.per * kHalfLn2, x2 = x * x;
  return fmaf(s * x2, fmaf(x2, fmaf(x2, fmaf(x2, kCap4, kCap3), kCap2), kCap1), s);
}
__device__ __forceinline__ float cap_large(float s, const Cap& c) {
  const float y = s * c.per;
  return fabsf(y) < kCapSeries ? cap_series(s, c) : c.top * fmaf(-2.f, rcp(1.f + ex2(y)), 1.f);
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

// Log probabilities of given tokens, with entropy and top alternatives.
//
//   x = scale * logit;  lse = m + log sum e^(x - m)
//   logp = x[target] - lse;  H = log sum e^(x - m) - sum (x - m) e^(x - m) / sum e^(x - m)
//
// One pass over the logits: near their bytes with 32-bit logits.  With bf16 neither the
// bytes (52% of the DRAM's peak) nor the issue slots (60%) are used up: a warp's loads and
// its arithmetic take turns, and waiting for a chunk's loads is the largest stall, barriers
// the next.  A thread
// keeps a running maximum m of the logits, s = sum 2^y and t = sum y 2^y over its
// elements, with y = (logit - m) scale log2 e; where y falls by d, s becomes 2^-d s and t
// becomes 2^-d (t - d s).  The difference comes first: logits of any size and scales of
// any size overflow nowhere but towards weight 0.
//
// Top alternatives.  Logit and index make one key, larger for a larger logit and
// for the smaller index of equal ones, so that all keys differ.  From the first
// chunk of a row the CTA takes a bound that at least top_k keys reach: the top_k-th
// of 32 groups' largest.  After that only what reaches the bound, a few hundred
// elements of a row, is collected in shared memory and ranked at the end, each key by
// counting those above it; every eight chunks the ones collected so far give a better
// bound (4: 53.2 / 156.7 us for the two below, 16: 53.4 / 160.3).  The groups' bound is
// the looser, the more keys are asked for: from eight on the first looks come after 1, 2
// and 4 chunks (twenty tokens of the rows below: 90.5 -> 74.2 us, 209 -> 181; one or five:
// 52.8 -> 53.6, 155 -> 157).
//
// Where more than kBuffer elements reach the bound before it gets better (a row that
// rises, or whose first chunk is masked), the part is read again, once for each key:
// with the first 8192 logits at -infinity, 512 rows of 201088 take 404 us for the best
// token and 2055 for twenty, where others take 55 and 75; 2047 rows of 100352 in 32 bits 892
// and 4906 for 143 and 179; rising rows up to 2565 and 5205; one row 11.8 and 81 for 10.2
// and 12.5.
//
// Split.  A row is cut into chunks of 16 KB, the chunks of all rows form one line,
// and each CTA takes an equal stretch.  A row that lies in several stretches is
// written in parts, joined by a second kernel.
//
// Four CTAs an SM, without loads ahead: the other warps cover them (5 CTAs: 54.6 / 153.4 us
// for the two below, 6: 68.0 / 202; the next chunk's loads into registers, some spilled:
// 63.6 -> 65.2 and 161 -> 169, before ranking was cut down; two chunks ahead into shared
// memory, by bulk copies of 2 KB a warp: 73 / 211, by cp.async: 65 / 187).
//
// Measured (back to back in a graph): 512 rows of 201088 in bf16, the best token, 51.8 us
// (4.0 TB/s; 44 without any ranking); 2047 rows of 100352 in 32 bits, five
// tokens, 151 us (5.4 TB/s; 128 without ranking); one row of 128256 in bf16, twenty
// tokens, 10.0 us (two launches, a few dependent loads and barriers each).
#include "launch.h"
#include "common.cuh"

#include <cfloat>

namespace tt {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kMaxCtas = 1024;
constexpr int kBuffer = 2048;                   // keys that are collected
constexpr int kEarly = 8;                       // keys from which the first looks come early
constexpr int kCheck = 8;                       // chunks from one look at their number to the next
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kErrShape = 2;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A part of a row: maximum and sums of all its logits, its largest keys.
struct alignas(16) Part {
  float m, s, t, pad;
  uint64_t keys[kMaxTop];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Larger for a larger logit, and of equal ones for the smaller index; never 0.
// -0 counts as 0, NaN as the largest.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) {
  uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) u = 0x7fffffffu;
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return uint64_t(u) << 32 | (kAll - i);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t u = uint32_t(key >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int32_t id_of(uint64_t key) { return int32_t(kAll - uint32_t(key)); }

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(__ldcg(static_cast<const uint16_t*>(row) + i));
  return __ldcg(static_cast<const float*>(row) + i);
}

// How far y falls where the maximum rises from `from` to `to`; 2^-kFar is 0, and times a
// sum it is finite.
constexpr float kFar = 1000.f;
__device__ __forceinline__ float fall(float to, float from, float k) {
  return fminf((to - from) * k, kFar);
}

// Maximum and sums of the union.
struct Sums {
  float m, s, t;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float k) {
  Sums r;
  r.m = max_nan(a.m, b.m);
  const float da = fall(r.m, a.m, k), db = fall(r.m, b.m, k);
  const float fa = ex2(-da), fb = ex2(-db);
  r.s = a.s * fa + b.s * fb;
  r.t = (a.t - da * a.s) * fa + (b.t - db * b.s) * fb;
  return r;
}

// The union of the warp's, in every lane.
__device__ __forceinline__ Sums join_warp(Sums z, float k) {
  float m = z.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
  const float d = fall(m, z.m, k), f = ex2(-d);
  float s = z.s * f, t = (z.t - d * z.s) * f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(kAll, s, o);
    t += __shfl_xor_sync(kAll, t, o);
  }
  return {m, s, t};
}

// Row r's target (in the first thread, and if there are any), and its logit.
__device__ __forceinline__ int target_of(const LogprobArgs& a, int64_t r) {
  return threadIdx.x == 0 && a.logp ? __ldcg(a.targets + r) : -1;
}
template <bool BF16>
__device__ __forceinline__ float target_logit(const LogprobArgs& a, const void* row, int t) {
  return t >= 0 && t < a.vocab ? logit<BF16>(row, t) : 0.f;
}

// The results of row r from its sums and its largest keys (in shared memory); by a warp.
template <bool BF16>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t r, const Sums& z,
                                          const uint64_t* keys, int t, float x, int32_t* err) {
  // NaN unless the maximum is finite
  const float ls = logf(z.s) + (z.m - z.m);
  const int tid = threadIdx.x;
  if (tid == 0) {
    if (a.entropy) a.entropy[r] = ls - z.t / z.s * kLn2;
    if (a.logp) {
      float y = t < 0 ? 0.f : NAN;
      if (t >= a.vocab) flag_error(err, kErrShape);
      if (t >= 0 && t < a.vocab) y = fmaf(x - z.m, a.scale, -ls);
      a.logp[r] = y;
    }
  }
  if (tid < a.top) {
    a.top_ids[r * a.top + tid] = id_of(keys[tid]);
    if (a.top_logp) a.top_logp[r * a.top + tid] = fmaf(logit_of(keys[tid]) - z.m, a.scale, -ls);
  }
}

// The `top` largest of n keys in falling order, zeros behind them if there are fewer:
// each by the number of those above it.
__device__ __forceinline__ void rank_keys(const uint64_t* from, int n, int top, uint64_t* to) {
  for (int i = threadIdx.x; i < top; i += kThreads)
    if (i >= n) to[i] = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = from[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += from[j] > key;
    if (above < top) to[above] = key;
  }
}

// The largest keys of the elements [lo, hi) one after the other: where more of them
// reached the bound than can be collected.
template <bool BF16>
__device__ __noinline__ void keys_by_rounds(const void* row, int64_t lo, int64_t hi, int top,
                                            uint64_t* to, uint64_t* part) {
  uint64_t last = ~0ull;
  for (int k = 0; k < top; ++k) {
    uint64_t best = 0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const uint64_t key = key_of(logit<BF16>(row, i), uint32_t(i));
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(kAll, best, o);
      best = other > best ? other : best;
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = part[w] > best ? part[w] : best;
    last = best;
    if (threadIdx.x == 0) to[k] = best;
    __syncthreads();
  }
}

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void un2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Elements [i, i + 16 bytes) of a row, -infinity where they are outside of it.
template <bool BF16>
__device__ __noinline__ uint4 piece_at_end(const void* row, int64_t i, int64_t vocab) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(row);
      const int64_t i0 = i + 2 * e, i1 = i0 + 1;
      const uint32_t lo = i0 >= 0 && i0 < vocab ? __ldcg(p + i0) : 0xff80u;
      const uint32_t hi = i1 >= 0 && i1 < vocab ? __ldcg(p + i1) : 0xff80u;
      w[e] = lo | hi << 16;
    } else {
      const int64_t i0 = i + e;
      w[e] = i0 >= 0 && i0 < vocab ? __ldcg(static_cast<const uint32_t*>(row) + i0) : 0xff800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest key among `pieces` pieces of a row, from element i on and `step` apart;
// read again, which only threads without anything above -infinity do.
template <bool BF16>
__device__ __noinline__ uint64_t largest_key(const void* row, int64_t i, int pieces, int step,
                                             int64_t vocab) {
  uint64_t most = 0;
  for (int j = 0; j < pieces; ++j, i += step) {
    for (int e = 0; e < (BF16 ? 8 : 4); ++e) {
      if (i + e < 0 || i + e >= vocab) continue;
      const uint64_t key = key_of(logit<BF16>(row, i + e), uint32_t(i + e));
      most = key > most ? key : most;
    }
  }
  return most;
}

// The largest of a piece's logits.
template <bool BF16>
__device__ __forceinline__ float largest_of(const uint4& v) {
  if constexpr (BF16) {
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w)));
    return max_nan(__low2float(m2), __high2float(m2));
  } else {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

// A bit for each of a piece's logits that is not below `least`.
template <bool BF16>
__device__ __forceinline__ uint32_t not_below(const uint4& v, float least) {
  const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      bits |= uint32_t(!(__uint_as_float(ws[e] << 16) < least)) << (2 * e);
      bits |= uint32_t(!(__uint_as_float(ws[e] & 0xffff0000u) < least)) << (2 * e + 1);
    } else {
      bits |= uint32_t(!(__uint_as_float(ws[e]) < least)) << e;
    }
  }
  return bits;
}

// Element e of a thread's pieces, by halves of what is left.
template <bool BF16, int kVectors>
__device__ __forceinline__ float element(const uint4 (&x)[kVectors], int e) {
  const int at = BF16 ? e >> 1 : e;
  uint32_t w[4 * kVectors];
#pragma unroll
  for (int j = 0; j < kVectors; ++j) w[4 * j] = x[j].x, w[4 * j + 1] = x[j].y, w[4 * j + 2] = x[j].z, w[4 * j + 3] = x[j].w;
#pragma unroll
  for (int half = 2 * kVectors; half > 0; half /= 2) {
#pragma unroll
    for (int i = 0; i < half; ++i) w[i] = at & half ? w[i + half] : w[i];
  }
  return __uint_as_float(!BF16 ? w[0] : e & 1 ? w[0] & 0xffff0000u : w[0] << 16);
}

// Sums of a piece's weights and of y times weight, -infinity told from the lowest logit.
template <bool BF16>
__device__ __noinline__ float2 sums_of_piece(uint4 v, float m, float k) {
  const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
  float2 r{0.f, 0.f};
  auto add = [&](float x) {
    const float y = fmaxf((x - m) * k, -kFar), w = ex2(y);
    r.x += w;
    r.y = fmaf(y, w, r.y);
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      add(__uint_as_float(ws[e] << 16));
      add(__uint_as_float(ws[e] & 0xffff0000u));
    } else {
      add(__uint_as_float(ws[e]));
    }
  }
  return r;
}

// kVectors: 16-byte pieces a thread and chunk.
template <bool BF16, int kVectors>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    logprobs_kernel(const LogprobArgs a, int chunks, int64_t total, Part* parts, int32_t* err) {
  constexpr int kPer = BF16 ? 8 : 4;  // elements of a piece
  constexpr int kBytes = BF16 ? 2 : 4;
  constexpr int kChunk = kPer * kVectors * kThreads;
  __shared__ uint64_t buffer[kBuffer];
  __shared__ uint64_t best[kMaxTop];
  __shared__ uint64_t groups[32];
  __shared__ Sums sums[kWarps];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int64_t begin = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
  const float k = a.scale * kLog2e;
  const uint64_t k2 = f2(k, k);
  const float far = __fdiv_ru(kFar, k);  // kFar in logits

  for (int64_t at = begin; at < end;) {
    const int64_t r = at / chunks;
    const int c0 = int(at - r * chunks);
    const int c1 = end - at < chunks - c0 ? c0 + int(end - at) : chunks;
    at += c1 - c0;
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + r * a.stride * kBytes;
    // pieces are cut from the 16-byte boundary before the row on: element i of the row
    // is element i + shift of them
    const int shift = int(reinterpret_cast<uintptr_t>(row) & 15u) / kBytes;
    const int64_t mine0 = int64_t(tid) * kPer - shift;  // this thread's first element
    auto load = [&](int c, uint4 (&x)[kVectors]) {
      const int64_t i0 = int64_t(c) * kChunk + mine0;
      const int64_t low = int64_t(c) * kChunk - shift;
      if (low >= 0 && low + kChunk <= a.vocab) {
        const uint4* p = reinterpret_cast<const uint4*>(row + i0 * kBytes);
#pragma unroll
        for (int j = 0; j < kVectors; ++j) x[j] = __ldcg(p + j * kThreads);
      } else {  // one of the row's ends
        const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;
        uint32_t cut = 0;
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
          const int64_t i = i0 + int64_t(j) * kThreads * kPer;
          x[j] = make_uint4(none, none, none, none);
          if (i >= 0 && i + kPer <= a.vocab)
            x[j] = __ldcg(reinterpret_cast<const uint4*>(row + i * kBytes));
          else if (i < a.vocab && i + kPer > 0)
            cut |= 1u << j;
        }
        for (; cut; cut &= cut - 1u) {
          const int j = __ffs(cut) - 1;
          const uint4 v = piece_at_end<BF16>(row, i0 + int64_t(j) * kThreads * kPer, a.vocab);
#pragma unroll
          for (int e = 0; e < kVectors; ++e)
            if (e == j) x[e] = v;
        }
      }
    };
    // asked for early: with its logit two round trips, which a short row would wait for
    const int t = c0 == 0 && c1 == chunks ? target_of(a, r) : -1;
    float t_logit = 0.f;
    Sums z{-INFINITY, 0.f, 0.f};
    uint64_t bound = 0;
    float least = -INFINITY;  // the bound's logit
    bool whole = true;        // all that reached the bound was collected
    if (tid == 0) s_count = 0;
    uint4 x[kVectors];
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      load(c, x);
      if (c == c0) t_logit = target_logit<BF16>(a, row, t);
      // ---- the largest
      float top;
      if constexpr (BF16) {
        auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        __nv_bfloat162 m2 = two(x[0].x);
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
          if (j > 0) m2 = __hmax2_nan(m2, two(x[j].x));
          m2 = __hmax2_nan(__hmax2_nan(m2, two(x[j].y)), __hmax2_nan(two(x[j].z), two(x[j].w)));
        }
        top = max_nan(__low2float(m2), __high2float(m2));
      } else {
        top = __uint_as_float(x[0].x);
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
          if (j > 0) top = max_nan(top, __uint_as_float(x[j].x));
          top = max_nan(max_nan(top, __uint_as_float(x[j].y)),
                        max_nan(__uint_as_float(x[j].z), __uint_as_float(x[j].w)));
        }
      }
      // ---- the sums
      if (!(top <= z.m)) {
        const float d = fall(top, z.m, k), f = ex2(-d);
        z.t = (z.t - d * z.s) * f;
        z.s *= f;
        z.m = max_nan(z.m, top);
      }
      const float m = z.m == -INFINITY ? 0.f : z.m;
      const uint64_t m2 = f2(-m, -m);
      uint64_t s2 = 0, t2 = 0;
      // What is `far` below the maximum or more has no weight, and is taken for `low`:
      // -infinity times weight 0 is NaN.  Rounded down, so that no logit is taken for one
      // with weight.
      float low = __fsub_rd(m, far);
      if constexpr (BF16) low = __bfloat162float(__float2bfloat16_rd(low));
      low = fmaxf(low, BF16 ? __uint_as_float(0xff7f0000u) : -FLT_MAX);
      const float least_y = (low - m) * k;
      if (least_y <= -200.f && least_y >= -FLT_MAX) {
        auto add = [&](float lo, float hi) {
          const uint64_t y = mul2(add2(f2(lo, hi), m2), k2);
          un2(y, lo, hi);
          const uint64_t w = f2(ex2(lo), ex2(hi));
          s2 = add2(s2, w);
          t2 = fma2(y, w, t2);
        };
        if constexpr (BF16) {
          const __nv_bfloat162 low2 = __float2bfloat162_rn(low);
#pragma unroll
          for (int j = 0; j < kVectors; ++j) {
            const uint32_t ws[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 v =
                  __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]), low2);
              const uint32_t w = *reinterpret_cast<const uint32_t*>(&v);
              add(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < kVectors; ++j) {
            add(fmaxf(__uint_as_float(x[j].x), low), fmaxf(__uint_as_float(x[j].y), low));
            add(fmaxf(__uint_as_float(x[j].z), low), fmaxf(__uint_as_float(x[j].w), low));
          }
        }
      } else {  // the lowest finite logit has weight, or one step below the maximum is too far
#pragma unroll 1
        for (int j = 0; j < kVectors; ++j) {
          uint4 v = x[0];
#pragma unroll
          for (int e = 1; e < kVectors; ++e)
            if (e == j) v = x[e];
          const float2 part = sums_of_piece<BF16>(v, m, k);
          z.s += part.x;
          z.t += part.y;
        }
      }
      float lo, hi;
      un2(s2, lo, hi);
      z.s += lo + hi;
      un2(t2, lo, hi);
      z.t += lo + hi;
      // ---- the largest keys
      if (a.top > 0) {
        const int64_t i0 = int64_t(c) * kChunk + mine0;
        if (c == c0) {
          // A key of this thread's that is no larger than its largest: the largest logit,
          // with the last index of the first piece that has it (one of -infinity may lie
          // outside the row).
          uint64_t mine = 0;
          if (top == -INFINITY) {
            if (i0 < a.vocab) mine = largest_key<BF16>(row, i0, kVectors, kThreads * kPer, a.vocab);
          } else {
#pragma unroll
            for (int j = 0; j < kVectors; ++j) {
              const uint64_t key = key_of(largest_of<BF16>(x[j]),
                                          uint32_t(i0 + int64_t(j) * kThreads * kPer + kPer - 1));
              mine = key > mine ? key : mine;
            }
          }
          uint64_t group = mine;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(kAll, group, o);
            group = other > group ? other : group;
          }
          if ((lane & 7) == 0) groups[warp * 4 + lane / 8] = group;
          __syncthreads();
          // every warp ranks the groups for itself; those without elements have 0
          const uint64_t g = groups[lane];
          int above = 0;
#pragma unroll 8
          for (int o = 0; o < 32; ++o) above += groups[o] > g;
          const int owner = __ffs(__ballot_sync(kAll, above == a.top - 1)) - 1;
          bound = owner >= 0 ? __shfl_sync(kAll, g, owner) : 0;
          least = bound ? logit_of(bound) : -INFINITY;
        }
        // what reaches the bound goes into the buffer, as far as there is room
        if (!(top < least)) {
          uint32_t hits = 0;
#pragma unroll
          for (int j = 0; j < kVectors; ++j) hits |= not_below<BF16>(x[j], least) << (j * kPer);
          for (; hits; hits &= hits - 1u) {
            const int e = __ffs(hits) - 1;
            const int64_t i = i0 + int64_t(e / kPer) * kThreads * kPer + e % kPer;
            if (i < 0 || i >= a.vocab) continue;
            const uint64_t key = key_of(element<BF16>(x, e), uint32_t(i));
            if (key < bound) continue;
            const int n = atomicAdd(&s_count, 1);
            if (n < kBuffer) buffer[n] = key;
          }
        }
        const int done = c - c0 + 1;
        if ((done % kCheck == 0 || (a.top >= kEarly && (done & (done - 1)) == 0)) && c + 1 < c1) {
          __syncthreads();
          const int n = s_count;
          whole &= n <= kBuffer;
          if (n >= 2 * a.top + 8 && whole) {  // a better bound
            rank_keys(buffer, n, a.top, best);
            __syncthreads();
            for (int i = tid; i < a.top; i += kThreads) buffer[i] = best[i];
            if (tid == 0) s_count = a.top;
            bound = best[a.top - 1];
            least = logit_of(bound);
          }
          __syncthreads();
        }
      }
    }
    // ---- the part's end
    z = join_warp(z, k);
    if (lane == 0) sums[warp] = z;
    __syncthreads();
    if (a.top > 0) {
      const int n = s_count;
      if (whole && n <= kBuffer) {
        rank_keys(buffer, n, a.top, best);
      } else {
        int64_t lo = int64_t(c0) * kChunk - shift, hi = int64_t(c1) * kChunk - shift;
        lo = lo < 0 ? 0 : lo;
        hi = hi < a.vocab ? hi : a.vocab;
        keys_by_rounds<BF16>(row, lo, hi, a.top, best, groups);
      }
      __syncthreads();
    }
    if (warp == 0) {
      z = join_warp(lane < kWarps ? sums[lane] : Sums{-INFINITY, 0.f, 0.f}, k);
      if (c0 == 0 && c1 == chunks) {
        write_row<BF16>(a, r, z, best, t, t_logit, err);
      } else {
        Part* p = parts + blockIdx.x * 2 + (c0 == 0 ? 1 : 0);
        if (tid == 0) p->m = z.m, p->s = z.s, p->t = z.t;
        if (tid < a.top) p->keys[tid] = best[tid];
      }
    }
    __syncthreads();
  }
}

// Joins the parts of the rows that lie in several stretches: block b has the row
// that goes on from stretch b into the next, if it began in b.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    logprobs_join_kernel(const LogprobArgs a, int chunks, int64_t total, const Part* parts,
                         int32_t* err) {
  __shared__ uint64_t buffer[kMaxTop * kMaxTop];
  __shared__ uint64_t firsts[kMaxCtas];
  __shared__ uint64_t best[kMaxTop];
  __shared__ Sums sums[kWarps];
  __shared__ uint64_t s_bound;
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t ctas = gridDim.x + 1;
  const float k = a.scale * kLog2e;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int64_t edge = total * (blockIdx.x + 1) / ctas;  // between the stretches
  const int64_t r = edge / chunks, first = r * chunks;
  if (edge == first || first < total * blockIdx.x / ctas) return;
  // the stretch of the row's last chunk: the last that begins at or before it
  const int n = int(((first + chunks) * ctas + total - 1) / total) - 1 - int(blockIdx.x) + 1;
  auto part = [&](int i) { return parts + (int64_t(blockIdx.x) + i) * 2 + (i == 0 ? 1 : 0); };
  if (tid == 0) s_count = 0, s_bound = 0;
  const int t = target_of(a, r);
  const float t_logit = target_logit<BF16>(a, static_cast<const uint8_t*>(a.logits) + r * a.stride * (BF16 ? 2 : 4), t);
  Sums z{-INFINITY, 0.f, 0.f};
  for (int i = tid; i < n; i += kThreads) {
    const float4 p = __ldcg(reinterpret_cast<const float4*>(part(i)));
    if (a.top > 0) firsts[i] = __ldcg(part(i)->keys);
    z = join(z, Sums{p.x, p.y, p.z}, k);
  }
  z = join_warp(z, k);
  if (lane == 0) sums[warp] = z;
  __syncthreads();
  if (a.top > 0) {
    // What reaches the top_k-th largest of the parts' first keys is at most top_k keys
    // of top_k parts.
    if (n >= a.top) {
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t key = firsts[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
          const uint64_t other = firsts[j];
          above += other > key || (other == key && j < i);
        }
        if (above == a.top - 1) s_bound = key;
      }
    }
    __syncthreads();
    const uint64_t bound = s_bound;
    // a part a warp, a key a lane, four parts on their way
    for (int i0 = warp; i0 < n; i0 += 4 * kWarps) {
      uint64_t key[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kWarps;
        key[e] = i < n && firsts[i] >= bound && lane < a.top ? __ldcg(part(i)->keys + lane) : 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key[e] != 0 && key[e] >= bound) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kMaxTop * kMaxTop) buffer[at] = key[e];
        }
      }
    }
    __syncthreads();
    rank_keys(buffer, s_count < kMaxTop * kMaxTop ? s_count : kMaxTop * kMaxTop, a.top, best);
    __syncthreads();
  }
  if (warp != 0) return;
  z = join_warp(lane < kWarps ? sums[lane] : Sums{-INFINITY, 0.f, 0.f}, k);
  write_row<BF16>(a, r, z, best, t, t_logit, err);
}

// Chunks of a row, wherever it begins.
int64_t chunks_of(int64_t vocab, bool bf16, int vectors) {
  const int64_t per = bf16 ? 8 : 4;
  const int64_t chunk = per * vectors * kThreads;
  return (vocab + per - 1 + chunk - 1) / chunk;
}

template <bool BF16, int kVectors>
cudaError_t launch(const DeviceInfo& di, const LogprobArgs& a, cudaStream_t s, bool pdl) {
  const int chunks = int(chunks_of(a.vocab, BF16, kVectors));
  const int64_t total = a.rows * chunks;
  int64_t ctas = int64_t(di.sms) * kCtasPerSm;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (ctas > total) ctas = total;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  Part* parts = static_cast<Part*>(a.ws);
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, kVectors>, a, chunks, total,
                                         parts, di.error_word))
    return e;
  // rows of one chunk, or as many CTAs as divide the rows evenly: nothing to join
  if (chunks == 1 || ctas == 1 || a.rows % ctas == 0) return cudaSuccess;
  cfg.gridDim = dim3(unsigned(ctas - 1));
  cfg.numAttrs = 1;  // the join always follows programmatically
  return cudaLaunchKernelEx(&cfg, logprobs_join_kernel<BF16>, a, chunks, total,
                            static_cast<const Part*>(parts), di.error_word);
}

template <bool BF16>
cudaError_t launch(const DeviceInfo& di, const LogprobArgs& a, cudaStream_t s, bool pdl) {
  // Few rows: chunks of a quarter, so that more SMs have one (one row of 128256: 14.7 us with
  // whole ones, 10.0).
  if (a.rows * chunks_of(a.vocab, BF16, 4) <= di.sms) return launch<BF16, 1>(di, a, s, pdl);
  return launch<BF16, 4>(di, a, s, pdl);
}

}  // namespace

size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top) {
  // two parts a CTA
  (void)rows, (void)vocab, (void)top;
  const DeviceInfo* di = device_info();
  const int64_t ctas = di && di->sms * kCtasPerSm < kMaxCtas ? di->sms * kCtasPerSm : kMaxCtas;
  return size_t(ctas) * 2 * sizeof(Part);
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, bool bf16, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  return bf16 ? launch<true>(*di, a, s, pdl) : launch<false>(*di, a, s, pdl);
}

}  // namespace tt

// Attention of one new token per sequence over the paged cache.
//
//   z[h][t] = f(scale * q[h] . k[j][t]) + slope[h] * (t - p),  j = h / G
//   out[h]  = sum_t e^z v[j][t] / (sum_t e^z + e^sink[h])
//
// over the visible tokens t of each sequence, G = heads / kv_heads query
// heads per kv head.  Every K and V row is needed once, for its G heads, so
// the work is bound by the cache's bytes: the kernel is built to keep the
// pages streaming.
//
// Split.  A sequence's tokens are cut into tiles (64 or 128 tokens); all
// tiles of all (sequence, kv head) pairs form one line, and CTA c of the
// C = min(SMs, tiles) takes the c-th C-th of it, whatever the lengths are:
// no SM has more than one tile more than another, and the host needs to know
// no length (the same launch serves a graph whose lengths grow).  A pair
// whose tiles lie in several CTAs is joined by the last of them to finish
// (a counter in the workspace), from the parts in CTA order, so that the
// result does not depend on who comes last.
//
// Inside a CTA four warps copy, each whole tiles in turn, 16 bytes a lane
// (cp.async), into a swizzled layout that the fragment loads read without bank
// conflicts; a pair's queries come with its first tiles.  The ring spans pair
// boundaries, so the copies run on while a pair is finished.  (One TMA box per
// page and matrix costs as much for a page of 1 KB as for one of 16: the FP8
// batch below took 308 us that way; four warps that share every tile 134 to 140,
// whole tiles each 117, before the units of the weights were a head's.)  Two groups of four warps take the tiles in turn, 16
// (or 2 x 16) tokens a warp, each with its own running maximum, sum and output;
// a pair's end joins them in shared memory.  (Four groups, with half the
// registers each: 137 us where two took 117.)
//
// Products, on mma.sync m16n8k16 with the tokens (or dims) as the 16 rows and
// the heads as the 8 columns, so that up to 8 heads fill it:
//   S[token][head]  = K Q^T     O^T[dim][head] += V^T P^T
// The order of the dims inside a contraction is free as long as both sides
// agree, so K fragments are 16-byte pieces of the rows, and V^T fragments
// are byte permutes of 16-byte pieces of two rows; P moves from the score
// fragment to the B operand by a transposing movmatrix.  (tcgen05 would need
// 128 rows of queries for a product of at most 16, and K and V would pass
// shared memory all the same.)
//   bf16: exact products; P as bf16 high + low parts (2^-16), since a decode
//     step's output should not lose to the cache's own precision.  The high part
//     is the largest below P, so that the low one is above 0 and both take an
//     infinite value to the same infinity (0 * infinity is NaN).
//   FP8: codes become f16 exactly; q becomes f16 after an exact power-of-two
//     prescale per head (its elements keep 11 bits down to 2^-29 of the
//     largest); the scales multiply scores and weights in 32 bits; P * scale
//     is rounded once to f16 (2^-11, against 2^-4 for a code), in a unit per
//     head that follows the largest P * scale so far, not the largest scale: a
//     row of a large scale may have no weight, and one of a small scale all of
//     it.  The unit puts the largest between 2^11 and 2^12 and is moved when one
//     passes 2^15, so products down to 2^-25 of the largest keep their 11 bits,
//     and smaller ones are off by 2^-36 of it.  When the maximum rises the unit
//     shrinks with the old weights and O stays as it is.
//
// Measured (back to back in a graph): 64 ragged sequences up to 16384 tokens,
// 64 / 8 heads of 64, FP8 pages of 16: 113 us, 4.9 TB/s (without the products
// 100: issue slots are 47% busy, copies and products share them); 32 up to 8192,
// 16 / 4 heads of 128, bf16: 47 us, 5.4 TB/s (without the products 43.8); one
// of 32768 tokens, 64 / 8 heads of 64, bf16: 18.3 us, of which 5 until the first
// tile (lengths, table, page: three dependent loads) and 4 to write and join
// the parts; one of 333 tokens 7.7 us.  The slowest CTA ends 11% after the mean.
#include <cmath>
#include <type_traits>

#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGroupWarps = 4;
constexpr int kCopyWarps = 4;
constexpr int kCopiers = 32 * kCopyWarps;
constexpr int kMaxCtas = 1024;                // counters in the workspace
constexpr int kSmemMax = 227 * 1024;
constexpr int kConsumerBar = 1;
constexpr float kLeastUnit = 0x1p-126f;       // of an FP8 cache's P * scale: the smallest normal number

template <int D, int NH, bool FP8>
struct Plan {
  static constexpr int kEs = FP8 ? 1 : 2;
  static constexpr int kRow = D * kEs;                    // bytes of a cache row
  static constexpr int kGroups = 2;  // tiles in work at once
  static constexpr int kConsumers = kGroups * kGroupWarps * 32;
  static constexpr int kThreads = kConsumers + kCopiers;
  // registers a thread: 65,536 less the copying warps' share
  // (40: FP8 batch 125 us, 56: 114.8, 72: 113.2, 88: 116.2)
  static constexpr int kCopyRegs = 72;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kRegs = (kLaunchRegs * kThreads - kCopyRegs * kCopiers) / kConsumers / 8 * 8;
  // 16-token chunks per warp and tile: 32 KB of K and V a tile, or 16 KB
  // where the rows are 64 bytes
  static constexpr int kTm = kRow == 256 ? 1 : 2;
  static constexpr int kTok = 16 * kGroupWarps * kTm;
  static constexpr int kPart = kTok * kRow;               // K (or V) bytes of a tile
  static constexpr int kOffScale = 2 * kPart;
  static constexpr int kOffQ = kOffScale + (FP8 ? 2 * kTok * 4 : 0);
  static constexpr int kStage = kOffQ + 8 * NH * D * 2;   // K, V, scales, the pair's queries
  // A warp's result: its output fragments as float4 units [2 NH][D / 32][32
  // lanes], then the heads' maxima and sums.  Two sets of slots where they
  // fit, so that a pair's result is read while the next is worked on.
  static constexpr int kUnits = 2 * NH * D;
  static constexpr int kSlot = 4 * kUnits + 16 * NH;      // floats
  static constexpr int kWarps = kGroups * kGroupWarps;
  static constexpr int kSets = NH * D > 128 ? 1 : 2;
  static constexpr int kScratch = kSets * kWarps * kSlot * 4;
  // XOR of a 16-byte piece's number within its row: the eight lanes of one
  // shared-memory phase then read eight different bank groups, both where
  // they read two rows (K) and where they read four (V)
  __device__ static constexpr int swizzle(int r) { return kRow == 64 ? (r >> 1) & 3 : r & 7; }
  static constexpr int kFixed =
      1024 + kScratch + (2 * kPagedMaxBatch + 2) * 4 + 512;  // alignment, parts, line, barriers
  // A multiple of the groups and of the copying warps, so that a stage is
  // always the same group's and the same warp's: they then wait for every
  // phase of its barriers in turn.  (With a stage that changes hands, one that
  // is ahead can find the phase before last and take it for its own.)
  static constexpr int kUnit = kGroups > kCopyWarps ? kGroups : kCopyWarps;
  static constexpr int kRaw = (kSmemMax - kFixed) / kStage / kUnit * kUnit;
  static constexpr int kStages = kRaw > 12 ? 12 : kRaw;
  static constexpr int kSmem = kFixed + kStages * kStage;
  static_assert(kScratch / kSets >= (kConsumers > kUnits ? kConsumers : 0) * 24, "join");
  static_assert(kStages >= 4 && kStages % kGroups == 0 && kStages % kCopyWarps == 0, "ring");
};

// Floats of one CTA part: a slot as above.
constexpr int part_floats(int group, int D) {
  const int nh = group > 8 ? 2 : 1;
  return 8 * nh * D + 16 * nh;
}

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_stride;
  int group;
  float scale, softcap;
  int window;
  const float* slopes;
  const float* sinks;
  uint16_t* out;
  float* lse;
  int32_t* counters;
  float* parts;
  int32_t* err;
};

template <bool FP8>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FP8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four E4M3 codes -> two f16x2 (exact).
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, int h) {
  return __byte_perm(a, b, h ? 0x7632 : 0x5410);
}

// The largest bf16 value below x > 0 (32-bit pattern); 0 of 0, NaN of a NaN.
__device__ __forceinline__ uint32_t bf16_below(float x) {
  return (max(__float_as_uint(x), 1u) - 1u) & 0xffff0000u;
}

// 16 bytes to shared memory, past L1; counted by the thread's next
// copies_arrive.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
template <int kConsumers>
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync %0, %1;" ::"r"(kConsumerBar), "n"(kConsumers) : "memory");
}

// The barrier, and whether any of its threads says so.
template <int kConsumers>
__device__ __forceinline__ bool consumer_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(p)), "r"(kConsumerBar), "n"(kConsumers)
      : "memory");
  return r != 0;
}

// The line of tiles: sequence b has nt(b) tiles from tile t0(b) on for each
// kv head; prefix[b] counts the tiles before it over all kv heads.
struct Line {
  const int32_t* prefix;
  const int32_t* len;
  int kv_heads, window, tok;
  __device__ __forceinline__ int first_tile(int b) const {
    const int n = len[b];
    return window > 0 && n > window ? (n - window) / tok : 0;
  }
  __device__ __forceinline__ int tiles(int b) const {
    const int n = len[b];
    return n == 0 ? 0 : (n + tok - 1) / tok - first_tile(b);
  }
};

// Where a CTA stands on the line.
struct At {
  int b, j, tile;  // tile counted from the pair's first
};
__device__ __forceinline__ At find(const Line& L, int batch, int item) {
  int lo = 0, hi = batch;  // the last b with prefix[b] <= item and tiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.prefix[mid] <= item) lo = mid; else hi = mid;
  }
  const int rem = item - L.prefix[lo], nt = L.tiles(lo);
  return {lo, rem / nt, rem % nt};
}

template <int D, int NH, bool FP8, bool LARGE_CAP>
__global__ void __launch_bounds__(Plan<D, NH, FP8>::kThreads, 1)
    paged_decode_kernel(const PagedKv kv, const DecodeArgs a) {
  using P = Plan<D, NH, FP8>;
  constexpr int kTok = P::kTok, kTm = P::kTm;
  constexpr int kGroups = P::kGroups, kConsumers = P::kConsumers, kThreads = P::kThreads;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem;
  float* scratch = reinterpret_cast<float*>(smem + P::kStages * P::kStage);
  int32_t* prefix = reinterpret_cast<int32_t*>(scratch + P::kScratch / 4);
  int32_t* slen = prefix + kPagedMaxBatch + 2;
  uint64_t* full = reinterpret_cast<uint64_t*>(slen + kPagedMaxBatch);
  uint64_t* empty = full + P::kStages;
  uint32_t* mask = reinterpret_cast<uint32_t*>(empty + P::kStages);  // granules present, per stage
  int* flags = reinterpret_cast<int*>(mask + P::kStages);  // [0] last to finish, [1] gave up
  int32_t* wsum = reinterpret_cast<int32_t*>(scratch);  // scan partials, before the main loop

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 32 + 1);  // a copying warp's lanes and its word
      mbar_init(smem_u32(&empty[i]), kGroupWarps);
    }
    flags[1] = 0;
    fence_mbar_init();
  }
  pdl_allow_next_grid();
  // The lengths and the table come into L2 while the preceding kernel ends (it
  // may still write them: L2 is where writes land, so nothing stale is kept).
  if (warp >= kGroups * kGroupWarps) {
    const int pt = tid - kConsumers;
    for (int i = pt * 32; i < kv.batch; i += kCopiers * 32) prefetch_l2(kv.lens + i);
    const int64_t entries = int64_t(kv.batch) * kv.pages_per_seq;
    const int64_t each = (entries + gridDim.x - 1) / gridDim.x;
    for (int64_t i = each * blockIdx.x + pt * 32; i < each * (blockIdx.x + 1) && i < entries;
         i += kCopiers * 32)
      prefetch_l2(kv.page_table + i);
  }
  pdl_wait_prior_grid();

  // ---- the line: lengths and the exclusive scan of the tiles
  const Line L{prefix, slen, kv.kv_heads, a.window, kTok};
  {
    constexpr int kPer = (kPagedMaxBatch + kThreads - 1) / kThreads;
    int mine[kPer], sum = 0;
    const int per = (kv.batch + kThreads - 1) / kThreads;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      mine[i] = 0;
      if (i < per && b < kv.batch) {
        slen[b] = paged_len(kv, b, blockIdx.x == 0 ? a.err : nullptr);
        mine[i] = L.tiles(b) * kv.kv_heads;
      }
      sum += mine[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) wsum[warp] = run;
    __syncthreads();
    int base = run - sum;
    for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i < per && b < kv.batch) prefix[b] = base;
      base += mine[i];
    }
    if (tid == kThreads - 1) prefix[kv.batch] = base;
    __syncthreads();
  }
  const int64_t T = prefix[kv.batch];
  // a CTA has a tile for each of its groups at least: fewer CTAs, fewer parts
  const int64_t Tg = (T + kGroups - 1) / kGroups;
  const int64_t C = Tg < gridDim.x ? Tg : gridDim.x;
  const int i0 = blockIdx.x < C ? int(T * blockIdx.x / C) : 0;
  const int i1 = blockIdx.x < C ? int(T * (blockIdx.x + 1) / C) : 0;
  const int G = a.group, heads = G * kv.kv_heads;

  constexpr int kGran = kTok / 16;  // granules of 16 tokens in a tile: each lies within a page
  if (warp >= kGroups * kGroupWarps) {
    // ================================================= the copying warps
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kCopyRegs));
    if (i0 >= i1) return;
    // Lane l looks up granule l % kGran of tile l / kGran of a batch of
    // tiles, one batch ahead of the copies: no table entry is waited for in
    // the loop.  Each warp has the same batch.
    constexpr int kBatch = 32 / kGran;
    const int pw = warp - kGroups * kGroupWarps;
    int row;  // the granule's first row in the pool, or -1
    int query;  // the tile is its group's first of a pair: the pair's first query row, or -1
    auto look = [&](int base) {
      const int it = base + lane / kGran;
      row = query = -1;
      if (it < i1) {
        const At w = find(L, kv.batch, it);
        const int first = it - w.tile > i0 ? it - w.tile : i0;
        if (it - first < kGroups) query = w.b * kv.kv_heads + w.j;
        const int n = slen[w.b], t = (L.first_tile(w.b) + w.tile) * kTok + lane % kGran * 16;
        // granules wholly before the window or past the length are not copied
        if (t < n && (a.window == 0 || t + 16 > n - a.window)) {
          const int page = paged_page(kv, w.b, t, a.err);
          if (page >= 0) row = int(paged_row(kv, page, w.j, t));
        }
      }
    };
    // this lane's piece of a granule's i-th 512 bytes: row and swizzled place
    constexpr int kLr = P::kRow / 16;  // lanes a row
    const int lr = lane / kLr, lc = lane % kLr;
    look(i0);
    for (int base = i0; base < i1; base += kBatch) {
      const int my_row = row, my_query = query;
      look(base + kBatch);
      const uint32_t got = __ballot_sync(kFull, my_row >= 0);
      for (int x = 0; x < kBatch && base + x < i1; ++x) {
        const int idx = base + x - i0, st = idx % P::kStages;
        if (idx % kCopyWarps != pw) continue;
        bool ok = true;
        if (idx >= P::kStages)
          ok = mbar_wait_bounded(smem_u32(&empty[st]), uint32_t((idx / P::kStages - 1) & 1));
        if (!__all_sync(kFull, ok) || *static_cast<volatile int*>(&flags[1])) {
          if (lane == 0) {
            flag_error(a.err, kErrTimeout);
            *static_cast<volatile int*>(&flags[1]) = 1;
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          return;
        }
        const uint32_t have = (got >> (x * kGran)) & (kFull >> (32 - kGran));
        const uint32_t stage = smem_u32(ring + st * P::kStage);
#pragma unroll
        for (int gr = 0; gr < kGran; ++gr) {
          const int r = __shfl_sync(kFull, my_row, x * kGran + gr);
          if (r >= 0) {
            const int64_t from = int64_t(r) * P::kRow + lane * 16;
#pragma unroll
            for (int w = 0; w < 2; ++w) {  // K, V
              const uint8_t* src = static_cast<const uint8_t*>(w ? kv.v : kv.k) + from;
              const uint32_t dst = stage + w * P::kPart + gr * 16 * P::kRow;
#pragma unroll
              for (int i = 0; i < P::kRow / 32; ++i) {
                const int q = lr + i * (512 / P::kRow);
                copy16(dst + q * P::kRow + ((lc ^ P::swizzle(q)) << 4), src + i * 512);
              }
            }
          }
        }
        const int bj = __shfl_sync(kFull, my_query, x * kGran);
        if (bj >= 0) {
          const int b = bj / kv.kv_heads, j = bj - b * kv.kv_heads;
          const uint16_t* src = a.q + int64_t(b) * a.q_stride + int64_t(j) * G * D;
          for (int i = lane; i < G * D / 8; i += 32)
            copy16(stage + P::kOffQ + i * 16, src + i * 8);
        }
        if constexpr (FP8) {
          constexpr int kPieces = 8 * kGran;  // 16 bytes: 4 of K, 4 of V a granule
#pragma unroll
          for (int u = 0; u < kPieces / 32; ++u) {
            const int e = u * 32 + lane, gr = e >> 3, w = (e >> 2) & 1, q = e & 3;
            const int r = __shfl_sync(kFull, my_row, x * kGran + gr);
            if (r >= 0)
              copy16(stage + P::kOffScale + (w * kTok + gr * 16 + q * 4) * 4,
                     (w ? kv.v_scales : kv.k_scales) + int64_t(r) + q * 4);
          }
        }
        if (lane == 0) {
          mask[st] = have;
          mbar_arrive(smem_u32(&full[st]));
        }
        copies_arrive(smem_u32(&full[st]));
      }
    }
    return;
  }

  // ==================================================== the computing warps
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::kRegs));
  // sequences without a visible token: no tiles, but rows to write
  for (int b = blockIdx.x; b < kv.batch; b += gridDim.x)
    if (L.tiles(b) == 0)
      for (int e = tid; e < heads * D / 8; e += kConsumers) {
        reinterpret_cast<uint4*>(a.out + int64_t(b) * heads * D)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && e < heads)
          a.lse[int64_t(b) * heads + e] = a.sinks ? __ldcg(a.sinks + e) : -INFINITY;
      }
  if (i0 >= i1) return;
  const int g = lane >> 2, qd = lane & 3;
  const int grp = warp / kGroupWarps, gw = warp % kGroupWarps;
  constexpr int KP = P::kRow / 64;  // 16-byte pieces of a row per lane in the score product
  constexpr int QR = D / 8;         // registers of q per lane and head tile
  constexpr int MT = D / 16;        // 16-dim tiles of the output
  const Cap cap = cap_of(a.softcap);
  // from the product's units: to log2 units, or with a small cap to its y
  const float unit = kLog2e * (!LARGE_CAP && a.softcap > 0.f ? cap.per : 1.f);
  const bool plain = LARGE_CAP ? !a.slopes : !(a.softcap > 0.f) && !a.slopes;

  uint32_t pairs = 0;  // done so far
  At at = find(L, kv.batch, i0);
  for (int it = i0; it < i1;) {
    const int b = at.b, j = at.j, nt = L.tiles(b), k0 = at.tile;
    const int here = i1 - it < nt - k0 ? i1 - it : nt - k0;
    const int n = slen[b];
    const int lo = a.window > 0 && n > a.window ? n - a.window : 0;
    const int tok0 = L.first_tile(b) * kTok;

    // ---- Q^T fragments: head g + 8 nh, the dims of this lane's pieces
    uint32_t qf[NH][QR];
    float fac[NH][2], slope[NH][2];  // heads 8 nh + 2 qd + {0, 1}
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hc = 8 * nh + 2 * qd + e;
        slope[nh][e] = a.slopes && hc < G ? __ldcg(a.slopes + j * G + hc) * kLog2e : 0.f;
      }
    auto load_q = [&](const uint8_t* qs) {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        const int h = g + 8 * nh;
        const uint4* qp = reinterpret_cast<const uint4*>(qs + h * D * 2);
        if constexpr (FP8) {
          float m = 0.f;
          uint4 v[KP][2];
#pragma unroll
          for (int c = 0; c < KP; ++c) {
            const int pc = D == 128 ? 2 * qd + c : qd;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              v[c][e] = h < G ? qp[2 * pc + e] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                m = fmaxf(m, fmaxf(fabsf(bf16_bits_to_f32(word(v[c][e], i) & 0xffffu)),
                                   fabsf(bf16_bits_to_f32(word(v[c][e], i) >> 16))));
            }
          }
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
          // 2^ex stays a normal number; a row whose largest element is below
          // 2^-112 is brought up less far
          const int ex = min(f16_prescale_exponent(m), 126);
          const float up = __int_as_float((127 + ex) << 23);
#pragma unroll
          for (int c = 0; c < KP; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                qf[nh][8 * c + 4 * e + i] =
                    pack_f16x2_scaled(bf16_bits_to_f32(word(v[c][e], i) & 0xffffu),
                                      bf16_bits_to_f32(word(v[c][e], i) >> 16), up);
          const float down = __int_as_float((127 - ex) << 23);
          fac[nh][0] = a.scale * __shfl_sync(kFull, down, 8 * qd);
          fac[nh][1] = a.scale * __shfl_sync(kFull, down, 8 * qd + 4);
        } else {
#pragma unroll
          for (int c = 0; c < KP; ++c) {
            const int pc = 8 * (c >> 1) + 2 * qd + (c & 1);
            const uint4 v = h < G ? qp[pc] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[nh][4 * c + i] = word(v, i);
          }
          fac[nh][0] = fac[nh][1] = a.scale;
        }
        fac[nh][0] = fminf(fmaxf(fac[nh][0] * unit, -kFiniteMax), kFiniteMax);
        fac[nh][1] = fminf(fmaxf(fac[nh][1] * unit, -kFiniteMax), kFiniteMax);
      }
    };

    float mrun[NH][2], lsum[NH][2], o[NH][MT][4];
    [[maybe_unused]] float ou[NH][2];  // FP8: the units of o
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      mrun[nh][0] = mrun[nh][1] = -INFINITY;
      ou[nh][0] = ou[nh][1] = kLeastUnit;
      lsum[nh][0] = lsum[nh][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        o[nh][mt][0] = o[nh][mt][1] = o[nh][mt][2] = o[nh][mt][3] = 0.f;
    }

    // ---- one tile; FULLT: every token of it is visible
    auto tile = [&](auto full_tile, int st, int t0, uint32_t have) {
      constexpr bool FULLT = decltype(full_tile)::value;
      const uint8_t* kb = ring + st * P::kStage;
      const uint8_t* vb = kb + P::kPart;
      // 16-byte piece p of row r
      auto piece = [&](const uint8_t* base, int r, int p) {
        return base + r * P::kRow + ((p ^ P::swizzle(r)) << 4);
      };
      auto visible = [&](int r) {
        const int t = t0 + r;
        return t >= lo && t < n && ((have >> (r >> 4)) & 1u);
      };
      // scores sc[tm][nh]: tokens r0 + (g | g + 8) x heads 8 nh + 2qd + (0 | 1)
      float sc[kTm][NH][4];
#pragma unroll
      for (int tm = 0; tm < kTm; ++tm) {
        const int r0 = 16 * (tm * kGroupWarps + gw) + g;
        float s2[NH][4];  // a second chain of products: half the latency
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[tm][nh][e] = s2[nh][e] = 0.f;
#pragma unroll
        for (int c = 0; c < KP; ++c) {
          const int p = FP8 ? (D == 128 ? 2 * qd + c : qd) : 8 * (c >> 1) + 2 * qd + (c & 1);
          const uint4 x = *reinterpret_cast<const uint4*>(piece(kb, r0, p));
          const uint4 y = *reinterpret_cast<const uint4*>(piece(kb, r0 + 8, p));
          if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x0, x1, y0, y1;
              e4m3x4(word(x, i), x0, x1);
              e4m3x4(word(y, i), y0, y1);
#pragma unroll
              for (int nh = 0; nh < NH; ++nh)
                mma16816<true>(i & 1 ? s2[nh] : sc[tm][nh], x0, y0, x1, y1, qf[nh][8 * c + 2 * i],
                               qf[nh][8 * c + 2 * i + 1]);
            }
          } else {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              mma16816<false>(sc[tm][nh], x.x, y.x, x.y, y.y, qf[nh][4 * c], qf[nh][4 * c + 1]);
              mma16816<false>(s2[nh], x.z, y.z, x.w, y.w, qf[nh][4 * c + 2],
                              qf[nh][4 * c + 3]);
            }
          }
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[tm][nh][e] += s2[nh][e];
      }
      // the scales of this lane's tokens
      [[maybe_unused]] float vs[kTm][2];
      if constexpr (FP8) {
        const float* ss = reinterpret_cast<const float*>(vb + P::kPart);
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * (tm * kGroupWarps + gw) + g + 8 * e;
            const float ks = ss[r];
            vs[tm][e] = ss[kTok + r];
            if (!FULLT && !visible(r)) vs[tm][e] = 0.f;
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              sc[tm][nh][2 * e] *= ks;
              sc[tm][nh][2 * e + 1] *= ks;
            }
          }
      }
      // to log2 units, mask, running maximum and sum
      if constexpr (LARGE_CAP) {
        float far = 0.f;
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sc[tm][nh][e] *= fac[nh][e & 1];
              far = fmaxf(far, fabsf(sc[tm][nh][e]));
            }
        const bool large = __any_sync(kFull, far * cap.per >= kCapSeries);
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[tm][nh][e] =
                  large ? cap_large(sc[tm][nh][e], cap) : cap_series(sc[tm][nh][e], cap);
      }
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * (tm * kGroupWarps + gw) + g + 8 * (e >> 1);
            float v = LARGE_CAP ? sc[tm][nh][e] : sc[tm][nh][e] * fac[nh][e & 1];
            if (!plain) {
              if (!LARGE_CAP && a.softcap > 0.f) v = cap_small(v, cap);
              v = fmaf(slope[nh][e & 1], float(t0 + r - (n - 1)), v);
            }
            if (!FULLT && !visible(r)) v = -INFINITY;
            sc[tm][nh][e] = v;
            mx[e & 1] = fmaxf(mx[e & 1], v);
          }
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float m = mx[h];
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
          const float mn = fmaxf(mrun[nh][h], m);
          const float ms = mn == -INFINITY ? 0.f : mn;  // nothing visible so far
          alpha[h] = ex2(mrun[nh][h] - ms);
          mrun[nh][h] = mn;
          mx[h] = ms;
        }
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[tm][nh][e] = ex2(sc[tm][nh][e] - mx[e & 1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t = 0.f;
#pragma unroll
          for (int tm = 0; tm < kTm; ++tm) t += sc[tm][nh][h] + sc[tm][nh][h + 2];
          lsum[nh][h] = lsum[nh][h] * alpha[h] + t;
          if constexpr (FP8) ou[nh][h] *= alpha[h];
        }
        if constexpr (!FP8) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[nh][mt][0] *= alpha[0];
            o[nh][mt][1] *= alpha[1];
            o[nh][mt][2] *= alpha[0];
            o[nh][mt][3] *= alpha[1];
          }
        }
      }
      // FP8: weights times scales, in the heads' units
      if constexpr (FP8) {
        float top[NH][2], iu[NH][2];
        bool move = false;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t = 0.f;
#pragma unroll
            for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& w = sc[tm][nh][h + 2 * e];
                w *= vs[tm][e];
                t = fmaxf(t, fabsf(w));
              }
            top[nh][h] = t;
            iu[nh][h] = rcp(ou[nh][h]);  // (of less than kLeastUnit: not used)
            move |= ou[nh][h] < kLeastUnit || t * iu[nh][h] > 0x1p15f;
          }
        if (__any_sync(kFull, move)) {
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float t = top[nh][h];
              t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
              t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
              t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
              // the power of two in t (of infinity: 2^127), 2^11 of which are the unit
              t = fminf(__uint_as_float(__float_as_uint(t) & 0x7f800000u), 0x1p127f) * 0x1p-11f;
              t = fmaxf(fmaxf(t, ou[nh][h]), kLeastUnit);
              iu[nh][h] = rcp(t);
              f[h] = ou[nh][h] * iu[nh][h];
              ou[nh][h] = t;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[nh][mt][0] *= f[0];
              o[nh][mt][1] *= f[1];
              o[nh][mt][2] *= f[0];
              o[nh][mt][3] *= f[1];
            }
          }
        }
#pragma unroll
        for (int tm = 0; tm < kTm; ++tm)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[tm][nh][e] *= iu[nh][e & 1];
      }
      // O^T += V^T P^T
#pragma unroll
      for (int tm = 0; tm < kTm; ++tm) {
        uint32_t ph[NH][2];
        [[maybe_unused]] uint32_t pl[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          const float* c = sc[tm][nh];
          if constexpr (FP8) {
            ph[nh][0] = transpose8x8(f16x2(c[0], c[1]));
            ph[nh][1] = transpose8x8(f16x2(c[2], c[3]));
          } else {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = bf16_below(c[e]);
            ph[nh][0] = transpose8x8(halves(h[0], h[1], 1));
            ph[nh][1] = transpose8x8(halves(h[2], h[3], 1));
            pl[nh][0] = transpose8x8(
                bf16x2(c[0] - __uint_as_float(h[0]), c[1] - __uint_as_float(h[1])));
            pl[nh][1] = transpose8x8(
                bf16x2(c[2] - __uint_as_float(h[2]), c[3] - __uint_as_float(h[3])));
          }
        }
        const int rv = 16 * (tm * kGroupWarps + gw) + 2 * qd;
        const int rr[4] = {rv, rv + 1, rv + 8, rv + 9};
        if constexpr (FP8) {
          // lane g: dims D/8 * g + (0 .. D/8 - 1); tile mt: row g is dim
          // 2 mt of them, row g + 8 dim 2 mt + 1
          uint32_t w[4][D / 32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool ok = FULLT || visible(rr[i]);
            if constexpr (D == 128) {
              const uint4 x = ok ? *reinterpret_cast<const uint4*>(piece(vb, rr[i], g))
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int u = 0; u < 4; ++u) w[i][u] = word(x, u);
            } else {
              const uint2 x = ok ? *reinterpret_cast<const uint2*>(piece(vb, rr[i], g >> 1) +
                                                                   8 * (g & 1))
                                 : make_uint2(0u, 0u);
              w[i][0] = x.x;
              w[i][1] = x.y;
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int sel = (mt & 1) ? 0x7362 : 0x5140;  // bytes a, b of row 1 and 2 interleaved
            uint32_t a0, a1, a2, a3;
            e4m3x4(__byte_perm(w[0][mt >> 1], w[1][mt >> 1], sel), a0, a1);
            e4m3x4(__byte_perm(w[2][mt >> 1], w[3][mt >> 1], sel), a2, a3);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
              mma16816<true>(o[nh][mt], a0, a1, a2, a3, ph[nh][0], ph[nh][1]);
          }
        } else {
          constexpr int CH = D / 64;
          uint4 v[4][CH];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool ok = FULLT || visible(rr[i]);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
              v[i][ch] = ok ? *reinterpret_cast<const uint4*>(piece(vb, rr[i], g + 8 * ch))
                            : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // D = 64: rows g, g + 8 are dims 8g + 2mt, + 1; D = 128: dims
            // 8g + mt and 64 + 8g + mt
            uint32_t a0, a1, a2, a3;
            if constexpr (D == 64) {
              a0 = halves(word(v[0][0], mt), word(v[1][0], mt), 0);
              a1 = halves(word(v[0][0], mt), word(v[1][0], mt), 1);
              a2 = halves(word(v[2][0], mt), word(v[3][0], mt), 0);
              a3 = halves(word(v[2][0], mt), word(v[3][0], mt), 1);
            } else {
              const int w = mt >> 1, hf = mt & 1;
              a0 = halves(word(v[0][0], w), word(v[1][0], w), hf);
              a1 = halves(word(v[0][CH - 1], w), word(v[1][CH - 1], w), hf);
              a2 = halves(word(v[2][0], w), word(v[3][0], w), hf);
              a3 = halves(word(v[2][CH - 1], w), word(v[3][CH - 1], w), hf);
            }
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              mma16816<false>(o[nh][mt], a0, a1, a2, a3, ph[nh][0], ph[nh][1]);
              mma16816<false>(o[nh][mt], a0, a1, a2, a3, pl[nh][0], pl[nh][1]);
            }
          }
        }
      }
    };

    bool gave_up = false;
    for (int x = 0; x < here; ++x) {
      const int idx = (it - i0) + x;
      if (idx % kGroups != grp) continue;
      const int st = idx % P::kStages;
      if (!__all_sync(kFull, mbar_wait_bounded(smem_u32(&full[st]),
                                               uint32_t((idx / P::kStages) & 1)))) {
        if (lane == 0) {
          flag_error(a.err, kErrTimeout);
          *static_cast<volatile int*>(&flags[1]) = 1;
        }
        gave_up = true;
        break;
      }
      if (x < kGroups) load_q(ring + st * P::kStage + P::kOffQ);  // the group's first tile
      const uint32_t have = mask[st];
      const int t0 = tok0 + (k0 + x) * kTok;
      const uint32_t all = kFull >> (32 - kGran);
      if (t0 >= lo && t0 + kTok <= n && have == all)
        tile(std::true_type{}, st, t0, have);
      else if (have)
        tile(std::false_type{}, st, t0, have);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
    }

    // ---- the pair's end: join the warps
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = lsum[nh][h];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        lsum[nh][h] = l;
      }
      if constexpr (FP8) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nh][mt][e] *= ou[nh][e & 1];
      }
    }
    // Unit (hf, qi) of a lane: head 8 (hf / 2) + 2 qd + hf % 2, four
    // consecutive dims from first_dim(qi, g) on.
    constexpr int QI = D / 32;
    constexpr bool kSplitDims = !FP8 && D == 128;  // rows g, g + 8 are 64 dims apart
    auto first_dim = [](int qi, int gg) {
      return kSplitDims ? 8 * gg + 4 * (qi & 1) + 64 * (qi >> 1) : D / 8 * gg + 4 * qi;
    };
    float* set = scratch + (P::kSets > 1 ? pairs & 1 : 0) * (P::kWarps * P::kSlot);
    ++pairs;
    const bool one = here == 1;  // a single tile: only its group has anything
    const int w0 = one ? (it - i0) % kGroups * kGroupWarps : 0;
    const int nw = one ? kGroupWarps : P::kWarps;
    if (warp >= w0 && warp < w0 + nw) {
      float* slot = set + warp * P::kSlot;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int qi = 0; qi < QI; ++qi) {
            float4 v;
            if constexpr (kSplitDims) {
              const int up = 2 * (qi >> 1), mt = 4 * (qi & 1);
              v = make_float4(o[nh][mt][h + up], o[nh][mt + 1][h + up], o[nh][mt + 2][h + up],
                              o[nh][mt + 3][h + up]);
            } else {
              v = make_float4(o[nh][2 * qi][h], o[nh][2 * qi][h + 2], o[nh][2 * qi + 1][h],
                              o[nh][2 * qi + 1][h + 2]);
            }
            reinterpret_cast<float4*>(slot)[((2 * nh + h) * QI + qi) * 32 + lane] = v;
          }
          if (g == 0) {
            slot[4 * P::kUnits + 8 * nh + 2 * qd + h] = mrun[nh][h];
            slot[4 * P::kUnits + 8 * NH + 8 * nh + 2 * qd + h] = lsum[nh][h];
          }
        }
    }
    // a wait that gave up: no result and no arrival, decided by all together
    if (consumer_any<P::kConsumers>(gave_up)) return;
    const bool whole = k0 == 0 && here == nt;
    // the warps' values of unit u of head r
    auto joined = [&](int r, int u, float& M, float& Lq) {
      M = -INFINITY;
      for (int w = 0; w < nw; ++w) M = fmaxf(M, set[(w0 + w) * P::kSlot + 4 * P::kUnits + r]);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      Lq = 0.f;
      const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll 4
      for (int w = 0; w < nw; ++w) {
        const float* p = set + (w0 + w) * P::kSlot;
        const float f = ex2(p[4 * P::kUnits + r] - ms);
        const float4 v = reinterpret_cast<const float4*>(p)[u];
        s.x = fmaf(v.x, f, s.x);
        s.y = fmaf(v.y, f, s.y);
        s.z = fmaf(v.z, f, s.z);
        s.w = fmaf(v.w, f, s.w);
        Lq = fmaf(p[4 * P::kUnits + 8 * NH + r], f, Lq);
      }
      return s;
    };
    // final values from O, max (log2 units) and sum of head r
    auto finish = [&](int r, int u, float4 s, float M, float Lq) {
      const int h = j * G + r, ul = u & 31, qi = (u >> 5) % QI;
      const int64_t row = int64_t(b) * heads + h;
      const int d0 = first_dim(qi, ul >> 2);
      const float inv = close_row(M, Lq, a.sinks, h, d0 == 0 ? a.lse : nullptr, row);
      *reinterpret_cast<uint2*>(a.out + row * D + d0) =
          make_uint2(bf16x2(s.x * inv, s.y * inv), bf16x2(s.z * inv, s.w * inv));
    };
    // head of unit u
    auto head_of = [](int u) {
      const int hf = (u >> 5) / QI;
      return 8 * (hf >> 1) + 2 * (u & 3) + (hf & 1);
    };
    if (whole) {
      for (int u = tid; u < P::kUnits; u += kConsumers) {
        const int r = head_of(u);
        if (r >= G) continue;
        float M, Lq;
        const float4 s = joined(r, u, M, Lq);
        finish(r, u, s, M, Lq);
      }
    } else {
      const int64_t s0 = L.prefix[b] + int64_t(j) * nt;  // the pair's first item
      const int cf = int(((s0 + 1) * C - 1) / T);        // CTAs of its first and last items
      const int cl = int(((s0 + nt) * C - 1) / T);
      float* part = a.parts + (int64_t(blockIdx.x) * 2 + (k0 == 0)) * P::kSlot;
      for (int u = tid; u < P::kUnits; u += kConsumers) {
        const int r = head_of(u);
        if (r >= G) continue;
        float M, Lq;
        const float4 s = joined(r, u, M, Lq);
        reinterpret_cast<float4*>(part)[u] = s;
        if (first_dim((u >> 5) % QI, (u & 31) >> 2) == 0) {
          part[4 * P::kUnits + r] = M;
          part[4 * P::kUnits + 8 * NH + r] = Lq;
        }
      }
      __threadfence();
      consumer_sync<P::kConsumers>();
      if (tid == 0) flags[0] = atomicAdd(a.counters + cf, 1) == cl - cf;
      consumer_sync<P::kConsumers>();
      if (flags[0]) {
        __threadfence();
        const int np = cl - cf + 1;
        // Each thread one unit: the parts in turn with the running maximum,
        // kJoin parts' loads in flight.  Where there are more threads than
        // units, kSub of them share a unit's parts and are joined after.
        constexpr int kJoin = 16;
        constexpr int kSub = kConsumers > P::kUnits ? kConsumers / P::kUnits : 1;
        for (int u0 = tid; u0 < P::kUnits * kSub; u0 += kConsumers) {
          const int u = u0 % P::kUnits, sub = u0 / P::kUnits, r = head_of(u);
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          float M = -INFINITY, Lq = 0.f;
          for (int p0 = sub; p0 < np && r < G; p0 += kJoin * kSub) {
            float4 v[kJoin];
            float m[kJoin], l[kJoin], mx = M;
#pragma unroll
            for (int e = 0; e < kJoin; ++e) {
              const int p = p0 + e * kSub;
              const bool in = p < np;
              const float* pp = a.parts + (int64_t(cf + (in ? p : 0)) * 2 + (!in || p == 0)) * P::kSlot;
              v[e] = in ? __ldcg(reinterpret_cast<const float4*>(pp) + u)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
              m[e] = in ? __ldcg(pp + 4 * P::kUnits + r) : -INFINITY;
              l[e] = in ? __ldcg(pp + 4 * P::kUnits + 8 * NH + r) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < kJoin; ++e) mx = fmaxf(mx, m[e]);
            const float ms = mx == -INFINITY ? 0.f : mx;
            const float old = ex2(M - ms);
            M = mx;
            s.x *= old;
            s.y *= old;
            s.z *= old;
            s.w *= old;
            Lq *= old;
#pragma unroll
            for (int e = 0; e < kJoin; ++e) {
              const float f = ex2(m[e] - ms);
              s.x = fmaf(v[e].x, f, s.x);
              s.y = fmaf(v[e].y, f, s.y);
              s.z = fmaf(v[e].z, f, s.z);
              s.w = fmaf(v[e].w, f, s.w);
              Lq = fmaf(l[e], f, Lq);
            }
          }
          if constexpr (kSub > 1) {
            // [sub][unit] values, then maxima, then sums, in the slots
            float4* sv = reinterpret_cast<float4*>(set);
            float* sm = set + 4 * kSub * P::kUnits;
            sv[u0] = s;
            sm[u0] = M;
            sm[kSub * P::kUnits + u0] = Lq;
            consumer_sync<P::kConsumers>();
            if (sub == 0) {
              float mx = M;
              for (int e = 1; e < kSub; ++e) mx = fmaxf(mx, sm[e * P::kUnits + u]);
              const float ms = mx == -INFINITY ? 0.f : mx;
              s = make_float4(0.f, 0.f, 0.f, 0.f);
              Lq = 0.f;
              for (int e = 0; e < kSub; ++e) {
                const float f = ex2(sm[e * P::kUnits + u] - ms);
                const float4 v = sv[e * P::kUnits + u];
                s.x = fmaf(v.x, f, s.x);
                s.y = fmaf(v.y, f, s.y);
                s.z = fmaf(v.z, f, s.z);
                s.w = fmaf(v.w, f, s.w);
                Lq = fmaf(sm[kSub * P::kUnits + e * P::kUnits + u], f, Lq);
              }
              M = mx;
            }
          }
          if (sub == 0 && r < G) finish(r, u, s, M, Lq);
        }
        if (tid == 0) a.counters[cf] = 0;  // ready for the next call
      }
    }
    if (P::kSets == 1) consumer_sync<P::kConsumers>();  // the slots are free again
    it += here;
    at.tile = 0;
    if (k0 + here == nt) {
      if (++at.j == kv.kv_heads) {
        at.j = 0;
        do ++at.b;
        while (at.b < kv.batch && L.tiles(at.b) == 0);
      }
    }
  }
}

template <int D, int NH, bool FP8, bool LARGE_CAP>
cudaError_t launch_as(const DeviceInfo& di, const PagedKv& kv, const PagedAttnArgs& a,
                      cudaStream_t s, bool pdl) {
  using P = Plan<D, NH, FP8>;
  auto kern = paged_decode_kernel<D, NH, FP8, LARGE_CAP>;
  static const bool fits = has_registers(kern, P::kLaunchRegs);
  if (!fits) return cudaErrorInvalidDeviceFunction;
  if (cudaError_t e = ensure_smem(di, kern, P::kSmem)) return e;
  // one CTA per SM, or one per tile that the table could hold where that is less
  const int64_t most =
      ((int64_t(kv.pages_per_seq) << kv.page_shift) + P::kTok - 1) / P::kTok * kv.batch *
      kv.kv_heads;
  int64_t grid = di.sms < kMaxCtas ? di.sms : kMaxCtas;
  if (grid > most) grid = most;
  DecodeArgs d;
  d.q = a.q;
  d.q_stride = a.q_stride;
  d.group = a.heads / kv.kv_heads;
  d.scale = a.scale;
  d.softcap = a.softcap;
  d.window = a.window;
  d.slopes = a.slopes;
  d.sinks = a.sinks;
  d.out = a.out;
  d.lse = a.lse;
  d.counters = static_cast<int32_t*>(a.ws);
  d.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kMaxCtas * 4);
  d.err = di.error_word;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, kv, d);
}

template <int D, int NH, bool FP8>
cudaError_t launch(const DeviceInfo& di, const PagedKv& kv, const PagedAttnArgs& a,
                   cudaStream_t s, bool pdl) {
  return a.softcap > kCapSmall ? launch_as<D, NH, FP8, true>(di, kv, a, s, pdl)
                               : launch_as<D, NH, FP8, false>(di, kv, a, s, pdl);
}

}  // namespace

size_t paged_decode_workspace_bytes(int group, int head_dim) {
  const DeviceInfo* di = device_info();
  const int64_t ctas = di && di->sms < kMaxCtas ? di->sms : kMaxCtas;
  return size_t(kMaxCtas) * 4 + size_t(ctas) * 2 * part_floats(group, head_dim) * 4;
}

cudaError_t launch_paged_decode(const PagedKv& kv, int head_dim, bool fp8,
                                const PagedAttnArgs& a, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  const bool wide = a.heads / kv.kv_heads > 8;
  if (head_dim == 64) {
    if (fp8)
      return wide ? launch<64, 2, true>(*di, kv, a, s, pdl) : launch<64, 1, true>(*di, kv, a, s, pdl);
    return wide ? launch<64, 2, false>(*di, kv, a, s, pdl) : launch<64, 1, false>(*di, kv, a, s, pdl);
  }
  if (fp8)
    return wide ? launch<128, 2, true>(*di, kv, a, s, pdl) : launch<128, 1, true>(*di, kv, a, s, pdl);
  return wide ? launch<128, 2, false>(*di, kv, a, s, pdl) : launch<128, 1, false>(*di, kv, a, s, pdl);
}

}  // namespace tt

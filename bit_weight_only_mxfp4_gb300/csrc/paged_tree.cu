// Attention of a tree of drafted tokens over the paged cache.
//
//   z[r][t] = f(scale * q[r] . k[j][t]) + slope[h] * (place of t - place of r)
//   out[r]  = sum_t e^z v[j][t] / (sum_t e^z + e^sink[h])
//
// A row r is one new token and one of the G query heads of kv head j.  It sees
// the cached tokens (within the window) and the new ones that its mask row names.
// A few new tokens read a long past, so the work is bound by the cache's bytes up
// to about 280 rows a kv head (140 on an FP8 cache), and by the products beyond;
// the products belong to the tensor cores either way:
//   S = Q K^T   128 rows x 128 tokens, tcgen05.mma, accumulator in TMEM
//   P = 2^(S - m) in bf16, back to TMEM
//   O += P V    A operand P from TMEM, B operand V as it lies in the cache
//
// Split.  A piece is a row tile (floor(128 / G) tokens x G heads) of a sequence and
// kv head; it has ceil(length / 128) K / V tiles.  The tiles of all pieces form
// one line, of which each CTA takes an equal stretch, whatever the lengths are.  A
// piece that lies in several CTAs is written in parts, joined in order by a second
// kernel.
//
// Inside a CTA the tiles of a piece go in turn to two groups of four warps, each
// with its own maximum, sum and O: while one group turns its scores into weights,
// the other's products run.  At the end of a piece (or of its part) both groups
// read both O's, half of the dims each.  (With one row tile for each group, as in
// the prompt kernel, a piece of one row tile would leave a group idle.)
//   warps 0-3, 4-7  softmax of the even and the odd tiles, one thread a row
//   warp 8          the products, issued by the warp in step, one elected lane
//   warp 9          the copies (TMA: one box per page and 64 dims; FP8: bulk
//                   copies of codes and scales)
//   warps 10, 11    make the V tiles safe (below); FP8: warps 10-15, which
//                   also turn E4M3 pages into bf16 tiles
// The running maximum is only raised (and O rescaled) when a row's maximum has
// grown by more than 2^8.
//
// Rounding.  Q and K products are exact, sums 32-bit; P is rounded once to bf16
// (2^-8 of each weight); the sum of weights is taken from the unrounded ones.
// FP8: codes become bf16 exactly, the scales multiply S and P in 32 bits.
//
// Masked values.  0 * NaN is NaN, so where the mask cuts a tile (the new tokens'
// tiles, the window's first ones) or pages are missing, V rows of no token are
// zeroed, elements that are not finite too, and the rows that do see them get
// them added at the end.  Tiles that all rows see whole need nothing of it.
#include <cmath>
#include <type_traits>

#include "paged_mma.cuh"

namespace tt {
namespace {

constexpr int kMmaWarp = 8, kLoadWarp = 9, kFixWarp = 10;
constexpr int kMaxCtas = 1024;
constexpr int kCounters = 1024;  // the decode kernel's, at the workspace's start: left alone
constexpr int kDirty = 16;

template <int D, bool FP8>
struct Plan {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kFixers = kThreads - 32 * kFixWarp;
  // registers a thread: at launch, of the softmax warps, of the others
  static constexpr int kLaunchRegs = FP8 ? 128 : 168;
  static constexpr int kSoftmaxRegs = FP8 ? 208 : 224;
  static constexpr int kOtherRegs = FP8 ? 48 : 56;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs,
                "register shares");
  static constexpr int kHalves = D / 64;            // 128-byte spans of a bf16 row
  static constexpr int kSpan = kKeys * 128;         // bytes of a tile's one span
  static constexpr int kTile = kSpan * kHalves;     // a K or V tile, or a Q tile
  static constexpr int kSlots = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int kRaw = FP8 ? kKeys * D + 2 * kKeys * 4 : 0;  // codes, both scales (with K)
  static constexpr int kRaws = FP8 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kOffKv = 2 * kTile;                      // (two Q tiles before)
  static constexpr int kOffRaw = kOffKv + kSlots * kTile;
  static constexpr int kOffScale = kOffRaw + kRaws * kRaw;      // [4 tiles][key, value][128]
  static constexpr int kOffDepth = kOffScale + (FP8 ? 4 * 2 * kKeys * 4 : 0);  // [2][2][128] floats
  static constexpr int kOffStat = kOffDepth + 4 * kKeys * 4;    // [2][128] maximum and sum
  static constexpr int kOffLine = kOffStat + 2 * kRows * 8;     // int64 [batch + 1]
  static constexpr int kOffStart = kOffLine + (kPagedMaxBatch + 2) * 8;
  static constexpr int kOffCount = kOffStart + kPagedMaxBatch * 4;
  static constexpr int kOffLen = kOffCount + kPagedMaxBatch * 4;
  static constexpr int kOffBar = kOffLen + kPagedMaxBatch * 4;
  static constexpr int kSmem = 1024 + kOffBar + 768;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOffBar % 8 == 0 && kOffLine % 8 == 0, "alignment");
  // TMEM columns of the groups: S, O and P.  With 128 dims P lies over S and the
  // next scores wait for P V; with 64 it has its own, and they wait only until S
  // is read.
  static constexpr bool kOwnP = D == 64;
  __host__ __device__ static constexpr int kColS(int g) { return 128 * g; }
  __host__ __device__ static constexpr int kColO(int g) { return 256 + D * g; }
  __host__ __device__ static constexpr int kColP(int g) { return kOwnP ? 384 + 64 * g : kColS(g); }
  static constexpr int kPartFloats = kRows * (D + 2);
};

struct KernelArgs {
  const int32_t* starts;
  int64_t tokens;
  int group, per_tile;  // heads per kv head, tokens per row tile
  float scale, softcap;
  int window;
  const float* slopes;
  const float* sinks;
  const uint32_t* masks;
  int words;
  uint16_t* out;
  float* lse;
  int4* joins;   // a record for each CTA whose last piece goes on in the next one's
  float* parts;  // [CTA][2]: of a piece that began before, of one that goes on
  int32_t* err;
};

// A CTA's part of a piece: K / V tiles [k0, k1) of the row tile that begins at
// flat token tok0.
struct Segment {
  int b, j, len, past;
  int tok0, i0, rows;  // the row tile's first token, its number, its tokens
  int most;            // new tokens that masks can name
  int lo;              // tokens that some row may see are in [lo, len)
  int all_lo, all_hi;  // tokens that every row sees
  int k0, k1;
  bool begins, ends;   // the piece
};

// The mask row's words of the sequence's `most` tokens.
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int w, int most) {
  const int n = most - 32 * w;
  if (n <= 0) return 0u;
  const uint32_t m = __ldcg(row + w);
  return n >= 32 ? m : m & ((1u << n) - 1u);
}
__device__ __forceinline__ int depth_of(const uint32_t* row, int most) {
  int n = 0;
  for (int w = 0; 32 * w < most; ++w) n += __popc(mask_word(row, w, most));
  return n > 0 ? n - 1 : 0;
}

// What a row sees: cached tokens [lo, past), new ones by its mask.
struct Sight {
  const uint32_t* mask;  // its row; nullptr: nothing
  const uint32_t* rows;  // the first row of the sequence
  int words, most, past, len, lo, window, depth;
  __device__ __forceinline__ bool sees(int t) const {
    if (!mask) return false;
    if (t < past) return t >= lo;
    const int k = t - past;
    if (t >= len || k >= most || !((__ldcg(mask + (k >> 5)) >> (k & 31)) & 1u)) return false;
    return window <= 0 || depth - depth_of(rows + int64_t(k) * words, most) < window;
  }
};

// Which of the 32 dims from d0 on have a value of +infinity, -infinity, NaN (a bit
// each) among the tokens of the tiles [k0, k1) that the row sees, in those tiles
// whose values were kept out of the product.
template <int D, bool FP8>
__device__ __noinline__ uint3 tree_not_finite(const PagedKv& kv, const Sight& s, int b, int j, int k0,
                                              int k1, int all_lo, int all_hi, bool holes, int d0) {
  uint3 x = make_uint3(0u, 0u, 0u);
  const int rows = 1 << kv.page_shift;
  for (int kt = k0; kt < k1; ++kt) {
    const int t0 = kt * kKeys;
    if (t0 >= all_lo && t0 + kKeys <= all_hi) {
      bool whole = true;
      for (int t = t0; holes && t < t0 + kKeys; t += rows) whole &= paged_page(kv, b, t, nullptr) >= 0;
      if (whole) continue;
    }
    for (int tp = t0; tp < t0 + kKeys && tp < s.len; tp += rows) {
      const int page = paged_page(kv, b, tp, nullptr);
      if (page < 0) continue;
      for (int t = tp; t < tp + rows && t < s.len; ++t) {
        if (!s.sees(t)) continue;
        const int64_t at = paged_row(kv, page, j, t);
        const uint8_t* src = static_cast<const uint8_t*>(kv.v) + (at * D + d0) * (FP8 ? 1 : 2);
        if constexpr (FP8) {
          if (!(fabsf(__ldcg(kv.v_scales + at)) <= kFiniteMax)) x.z = kAll;
          for (int d = 0; d < 32; d += 4) {
            const uint32_t v = __ldcg(reinterpret_cast<const uint32_t*>(src + d));
            for (int e = 0; e < 4; ++e) x.z |= uint32_t(((v >> (8 * e)) & 0x7fu) == 0x7fu) << (d + e);
          }
        } else {
          for (int d = 0; d < 32; d += 2) {
            const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(src + 2 * d));
            for (int e = 0; e < 2; ++e) {
              const uint32_t v = (w >> (16 * e)) & 0xffffu;
              x.x |= uint32_t(v == 0x7f80u) << (d + e);
              x.y |= uint32_t(v == 0xff80u) << (d + e);
              x.z |= uint32_t((v & 0x7fffu) > 0x7f80u) << (d + e);
            }
          }
        }
      }
    }
  }
  return x;
}

// What is done to the scores: nothing but a positive scale; a cap, a bias or
// another scale; a large cap.
enum Scores { kPlain, kGeneral, kLargeCap };
template <int D, bool FP8, Scores SC>
__global__ void __launch_bounds__(Plan<D, FP8>::kThreads, 1)
    paged_tree_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ PagedKv kv, const KernelArgs a) {
  using P = Plan<D, FP8>;
  constexpr bool GEN = SC != kPlain;
  constexpr int kThreads = P::kThreads, kFixers = P::kFixers;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + P::kOffScale);
  float* shifts = reinterpret_cast<float*>(smem + P::kOffDepth);
  float2* stat = reinterpret_cast<float2*>(smem + P::kOffStat);
  int64_t* line = reinterpret_cast<int64_t*>(smem + P::kOffLine);  // tiles before a sequence's
  int32_t* first = reinterpret_cast<int32_t*>(smem + P::kOffStart);
  int32_t* count = reinterpret_cast<int32_t*>(smem + P::kOffCount);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + P::kOffLen);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kOffBar);
  uint64_t* empty = full + P::kSlots;
  uint64_t* ready = empty + P::kSlots;   // slot made safe, or converted
  uint64_t* raw_full = ready + P::kSlots;
  uint64_t* raw_empty = raw_full + 4;
  uint64_t* q_full = raw_empty + 4;      // [2], of the Q tiles
  uint64_t* q_free = q_full + 2;         // [2]
  uint64_t* s_full = q_free + 2;         // [2], of the groups, and so on
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* s_read = o_done + 2;
  uint64_t* shifted = s_read + 2;
  uint64_t* posted = shifted + 2;        // both groups' maxima and sums
  uint64_t* taken = posted + 1;          // both groups' O's
  uint64_t* drained = taken + 1;
  uint32_t* have = reinterpret_cast<uint32_t*>(drained + 1);  // [8] boxes present, per tile
  int* dirty = reinterpret_cast<int*>(have + 8);              // [kDirty] segment number + 1
  int* misc = dirty + kDirty;  // [0] TMEM address, [1] quit, [2, 3] holes of the groups
  volatile int* quit = misc + 1;
  int64_t* scan = reinterpret_cast<int64_t*>(stat);  // [warps], before the main loop
  static_assert(kThreads / 32 * 8 <= 2 * kRows * 8, "scan");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P::kSlots; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
      mbar_init(smem_u32(&ready[i]), kFixers);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), kFixers);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&q_full[g]), 1);
      mbar_init(smem_u32(&q_free[g]), 2);
      mbar_init(smem_u32(&s_full[g]), 1);
      mbar_init(smem_u32(&p_full[g]), kRows);
      mbar_init(smem_u32(&o_done[g]), 1);
      mbar_init(smem_u32(&s_read[g]), kRows);
      mbar_init(smem_u32(&shifted[g]), kRows);
    }
    mbar_init(smem_u32(posted), 2 * kRows);
    mbar_init(smem_u32(taken), 2 * kRows);
    mbar_init(smem_u32(drained), 1);
    for (int i = 0; i < kDirty; ++i) dirty[i] = 0;
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&misc[0])),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_allow_next_grid();
  pdl_wait_prior_grid();

  // ---- the line: tiles of every sequence, scanned
  const int64_t tokens = a.tokens;
  const int G = a.group, heads = G * kv.kv_heads, TT = a.per_tile;
  auto start_of = [&](int b) {
    const int64_t s = __ldcg(a.starts + b);
    return int(s < 0 ? 0 : s > tokens ? tokens : s);
  };
  auto low_of = [&](int past) { return a.window > 0 && past + 1 > a.window ? past + 1 - a.window : 0; };
  auto tiles_of = [&](int b) {  // K / V tiles of a piece; one where there is no key, for the result
    const int n = (lens[b] + kKeys - 1) / kKeys - low_of(lens[b] - count[b]) / kKeys;
    return n > 0 ? n : 1;
  };
  auto row_tiles = [&](int b) { return (count[b] + TT - 1) / TT; };
  for (int b = tid; b < kv.batch; b += kThreads) {
    const int s0 = start_of(b), s1 = start_of(b + 1);
    first[b] = s0;
    count[b] = s1 > s0 ? s1 - s0 : 0;
    lens[b] = paged_len(kv, b, blockIdx.x == 0 ? a.err : nullptr);
  }
  __syncthreads();
  {
    constexpr int kPer = (kPagedMaxBatch + kThreads - 1) / kThreads;
    const int per = (kv.batch + kThreads - 1) / kThreads;
    int64_t mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      mine[i] = i < per && b < kv.batch ? int64_t(tiles_of(b)) * row_tiles(b) * kv.kv_heads : 0;
      sum += mine[i];
    }
    int64_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kAll, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) scan[warp] = run;
    __syncthreads();
    int64_t before = run - sum;
    for (int w = 0; w < warp; ++w) before += scan[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i < per && b < kv.batch) line[b] = before;
      before += mine[i];
    }
    if (tid == kThreads - 1) line[kv.batch] = before;
    fence_before();
    __syncthreads();
    fence_after();
  }
  const uint32_t tmem = uint32_t(misc[0]);
  // The CTA's stretch [begin, end) of the line: an equal share; two tiles at least,
  // one for each group.
  const int64_t total = line[kv.batch];
  const int sms = gridDim.x, cta = blockIdx.x;
  const int ctas = total >= 2 * sms ? sms : int((total + 1) / 2);
  const int64_t begin = cta < ctas ? total * cta / ctas : 0;
  const int64_t end = cta < ctas ? total * (cta + 1) / ctas : 0;

  // the piece that tile `at` of the line belongs to: its sequence, its first tile
  auto piece_at = [&](int64_t at, int& b, int& piece, int& tile) {
    int lo = 0, hi = kv.batch;  // the last b with line[b] <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (line[mid] <= at) lo = mid; else hi = mid;
    }
    b = lo;
    const int64_t rem = at - line[lo];
    const int nt = tiles_of(lo);
    piece = int(rem / nt);
    tile = int(rem - int64_t(piece) * nt);
  };
  auto segment_at = [&](int64_t at) {
    Segment w;
    int piece, tile;
    piece_at(at, w.b, piece, tile);
    const int rts = row_tiles(w.b), nt = tiles_of(w.b), n = count[w.b];
    w.j = piece / rts;
    w.i0 = (piece - w.j * rts) * TT;
    w.tok0 = first[w.b] + w.i0;
    w.rows = n - w.i0 < TT ? n - w.i0 : TT;
    w.len = lens[w.b];
    w.past = w.len - n;
    w.most = n < 32 * a.words ? n : 32 * a.words;
    w.lo = low_of(w.past);
    w.all_hi = w.past > 0 ? w.past : 0;
    // the deepest row's window
    w.all_lo = a.window > 0 && w.past + w.most > a.window ? w.past + w.most - a.window : 0;
    const int64_t left = end - at;
    w.k0 = w.lo / kKeys + tile;
    w.k1 = w.k0 + (left < nt - tile ? int(left) : nt - tile);
    w.begins = tile == 0;
    w.ends = left >= nt - tile;
    return w;
  };
  // the record of the piece that begins here and goes on in the next CTAs
  if (tid == 0 && a.joins) {
    int4 rec = make_int4(0, 0, 0, 0);
    if (end > begin) {
      int b, piece, tile;
      piece_at(end - 1, b, piece, tile);
      const int nt = tiles_of(b);
      const int64_t from = end - 1 - tile;
      if (from >= begin && from + nt > end) {
        const int last = int(((from + nt) * ctas + total - 1) / total) - 1;
        const int rts = row_tiles(b), i0 = (piece % rts) * TT, n = count[b] - i0;
        rec = make_int4(last - cta + 1, first[b] + i0, n < TT ? n : TT, piece / rts);
      }
    }
    a.joins[cta] = rec;
  }
  const int br_shift = kv.page_shift;  // rows of a box: a page, 16 .. 128
  const int boxes = kKeys >> br_shift;

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kOtherRegs));
    if (warp == kLoadWarp) {
      // ============================================================ copies
      uint32_t n = 0;   // slots used
      uint32_t seq = 0, asked = 0;  // segments, Q tiles
      uint32_t nt = 0;  // tiles
      bool ok = true;
      for (int64_t at = begin; ok && at < end; ++seq) {
        const Segment w = segment_at(at);
        at += w.k1 - w.k0;
        const uint32_t qb = seq & 1u;
        // a Q tile is free when the last score products of the segment are done
        if (seq >= 2)
          ok = __all_sync(kAll, wait(&q_free[qb], ((seq >> 1) - 1) & 1u, quit, a.err));
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&q_full[qb]);
          mbar_arrive_expect_tx(bar, uint32_t(TT * G * 128 * P::kHalves));
          for (int h = 0; h < P::kHalves; ++h)
            tma_q(sbase + qb * P::kTile + h * P::kSpan, &map_q, 64 * h, w.j * G, w.tok0, bar);
        }
        __syncwarp();
        ++asked;
        auto look = [&](int kt) {
          const int t = kt * kKeys + (lane << br_shift);
          const bool in = lane < boxes && t < w.len && t + (1 << br_shift) > w.lo;
          return in ? paged_page(kv, w.b, t, a.err) : -1;
        };
        int ahead = look(w.k0);
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++nt) {
          const int page = ahead;
          if (kt + 1 < w.k1) ahead = look(kt + 1);  // the next tile's, while this one is copied
          const uint32_t got = __ballot_sync(kAll, page >= 0);
          const int64_t row =
              page >= 0 ? paged_row(kv, page, w.j, kt * kKeys + (lane << br_shift)) : 0;
          const uint32_t bytes_row = 128u * P::kHalves;
          for (int part = 0; part < 2; ++part, ++n) {  // K, then V
            if constexpr (FP8) {
              const uint32_t s = n % P::kRaws, turn = n / P::kRaws;
              ok = turn == 0 || wait(&raw_empty[s], (turn - 1) & 1u, quit, a.err);
              ok = __all_sync(kAll, ok);
              if (!ok) break;
              const uint32_t bar = smem_u32(&raw_full[s]);
              if (lane == 0) {
                have[nt & 7u] = got;
                mbar_arrive_expect_tx(bar, __popc(got) * (uint32_t(part ? D : D + 8) << br_shift));
              }
              __syncwarp();
              if (page >= 0) {
                const uint32_t dst = sbase + P::kOffRaw + s * P::kRaw;
                const uint8_t* src = static_cast<const uint8_t*>(part ? kv.v : kv.k) + row * D;
                bulk_copy(dst + ((uint32_t(lane) * D) << br_shift), src, uint32_t(D) << br_shift,
                          bar);
                if (part == 0) {  // both scales with K: the softmax needs them after S
                  const uint32_t so = dst + kKeys * D + (uint32_t(lane) << (br_shift + 2));
                  bulk_copy(so, kv.k_scales + row, 4u << br_shift, bar);
                  bulk_copy(so + kKeys * 4, kv.v_scales + row, 4u << br_shift, bar);
                }
              }
            } else {
              const uint32_t s = n % P::kSlots, turn = n / P::kSlots;
              ok = turn == 0 || wait(&empty[s], (turn - 1) & 1u, quit, a.err);
              ok = __all_sync(kAll, ok);
              if (!ok) break;
              const uint32_t bar = smem_u32(&full[s]);
              if (lane == 0) {
                have[nt & 7u] = got;
                mbar_arrive_expect_tx(bar, __popc(got) * (bytes_row << br_shift));
              }
              __syncwarp();
              if (page >= 0) {
                const uint32_t dst =
                    sbase + P::kOffKv + s * P::kTile + (uint32_t(lane) << (br_shift + 7));
                for (int h = 0; h < P::kHalves; ++h)
                  tma_rows(dst + h * P::kSpan, part ? &map_v : &map_k, 64 * h, int(row), bar);
              }
            }
          }
        }
      }
      if (!ok) {  // gave up: the copies in flight land before the CTA ends
        uint64_t* f = FP8 ? raw_full : full;
        const uint32_t m = FP8 ? (P::kRaws ? P::kRaws : 1) : P::kSlots;
        for (uint32_t i = 1; i <= m && i <= n; ++i)
          (void)mbar_wait_bounded(smem_u32(&f[(n - i) % m]), ((n - i) / m) & 1u);
        for (uint32_t i = 1; i <= 2 && i <= asked; ++i)
          (void)mbar_wait_bounded(smem_u32(&q_full[(asked - i) & 1u]), ((asked - i) >> 1) & 1u);
      }
    } else if (warp == kMmaWarp) {
      // ========================================================== products
      // One warp for both groups, whichever is ready.  The commits free the slots,
      // so that a copy begins as soon as the products are through with its place.
      // Products finish in order, so scores that are there say that the P V issued
      // before them is done.
      const uint32_t kv0 = sbase + P::kOffKv;
      uint32_t n = 0, seq = 0, my0 = 0, my1 = 0;  // slots; segments; tiles of the groups
      bool ok = tmem == 0;  // all columns are ours, so they begin at 0
      if (!ok && lane == 0) {
        *quit = 1;
        flag_error(a.err, kErrShape);
      }
      auto scores = [&](auto gc, uint32_t slot) {
        constexpr int g = decltype(gc)::value;
        const uint64_t q = desc_k(sbase + (seq & 1u) * P::kTile), k = desc_k(kv0 + slot * P::kTile);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t off = ((i >> 2) * P::kSpan + (i & 3) * 32) >> 4;
          mma_ss(P::kColS(g), q + off, k + off, idesc(kKeys, false), i > 0);
        }
        commit(smem_u32(&s_full[g]));
        commit(smem_u32(&empty[slot]));
      };
      auto values = [&](auto gc, uint32_t slot, uint32_t more) {
        constexpr int g = decltype(gc)::value;
        const uint64_t v = desc_mn(kv0 + slot * P::kTile, P::kHalves > 1 ? P::kSpan : 1024);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(P::kColO(g), P::kColP(g) + 8 * k, v + k * (2048 >> 4),
                 idesc(D, true), k > 0 ? 1u : more);
      };
      auto key_bar = [&](uint32_t m) {
        return smem_u32(FP8 ? &ready[m % P::kSlots] : &full[m % P::kSlots]);
      };
      auto phase = [&](uint32_t m) { return (m / P::kSlots) & 1u; };
      using G0 = std::integral_constant<int, 0>;
      using G1 = std::integral_constant<int, 1>;
      for (int64_t at = begin; ok && at < end; ++seq) {
        const Segment w = segment_at(at);
        const uint32_t nk = __shfl_sync(kAll, w.k1 - w.k0, 0);
        at += nk;
        ok = __all_sync(kAll, wait(&q_full[seq & 1u], (seq >> 1) & 1u, quit, a.err));
        if (!ok) break;
        const uint32_t nk0 = (nk + 1) / 2, nk1 = nk / 2;
        // of each group: products P V issued, scores issued
        uint32_t v0 = 0, s0 = 0, v1 = 0, s1 = 0;
        uint64_t since = 0;  // of the idle stretch
        auto tile = [&](auto gc, uint32_t nkg, uint32_t& vi, uint32_t& si, uint32_t& my) {
          constexpr int g = decltype(gc)::value;
          bool did = false;
          const uint32_t m = n + 2 * (2 * vi + g);  // the tile's K
          if (vi < si) {
            const bool go =
                mbar_test_wait(smem_u32(&p_full[g]), my & 1u) &&
                mbar_test_wait(smem_u32(&ready[(m + 1) % P::kSlots]), phase(m + 1));
            if (__all_sync(kAll, go)) {
              fence_after();
              values(gc, (m + 1) % P::kSlots, vi > 0);
              commit(smem_u32(&empty[(m + 1) % P::kSlots]));
              if (P::kOwnP || vi + 1 == nkg) commit(smem_u32(&o_done[g]));
              ++vi;
              ++my;
              did = true;
            }
          }
          // the next scores: with 128 dims once the P V that lie there are issued,
          // else once those before are read (my - vi tiles were before this segment)
          if (si < nkg && (P::kOwnP || si == vi)) {
            const uint32_t ms = n + 2 * (2 * si + g);
            const bool go =
                (!P::kOwnP || mbar_test_wait(smem_u32(&s_read[g]), (my - vi + si - 1) & 1u)) &&
                mbar_test_wait(key_bar(ms), phase(ms));
            if (__all_sync(kAll, go)) {
              fence_after();
              scores(gc, ms % P::kSlots);
              ++si;
              did = true;
            }
          }
          return did;
        };
        for (uint32_t idle = 0; v0 < nk0 || v1 < nk1;) {
          bool did = tile(G0{}, nk0, v0, s0, my0);
          did |= tile(G1{}, nk1, v1, s1, my1);
          if (did) {
            idle = 0;
          } else if ((++idle & 63u) == 0u) {
            if (idle == 64u) since = globaltimer_ns();
            if (globaltimer_ns() - since > kWaitLimitNs && lane == 0) {
              *quit = 1;
              flag_error(a.err, kErrTimeout);
            }
            if (__any_sync(kAll, *quit)) {
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        n += 2 * nk;
      }
      // nothing of the tensor cores is under way when the CTA ends
      commit(smem_u32(drained));
      (void)mbar_wait_bounded(smem_u32(drained), 0);
      __syncwarp();
    } else if (warp >= kFixWarp) {
      // ===================================== V tiles made safe; FP8 -> bf16
      const int ft = tid - kFixWarp * 32;
      uint32_t n = 0, nt = 0;
      int seq = 0;
      bool ok = true;
      for (int64_t at = begin; ok && at < end;) {
        const Segment w = segment_at(at);
        at += w.k1 - w.k0;
        ++seq;
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++nt) {
          const int t0 = kt * kKeys;
          const bool cut = t0 < w.all_lo || t0 + kKeys > w.all_hi;
          for (int part = 0; part < 2; ++part, ++n) {
            const uint32_t s = n % P::kSlots, turn = n / P::kSlots;
            uint8_t* tile = smem + P::kOffKv + s * P::kTile;
            if constexpr (FP8) {
              const uint32_t rs = n % P::kRaws;
              ok = wait(&raw_full[rs], (n / P::kRaws) & 1u, quit, a.err) &&
                   (turn == 0 || wait(&empty[s], (turn - 1) & 1u, quit, a.err));
              if (!ok) break;
              const uint8_t* raw = smem + P::kOffRaw + rs * P::kRaw;
              const uint32_t got = have[nt & 7u];
              const uint32_t whole = kAll >> (32 - boxes);
              const bool sure = !cut && got == whole;
              bool bad = false;
              constexpr int kC = D / 16;  // 16-byte pieces of a raw row
              constexpr int kIlp = 4;  // pieces in work at once
#pragma unroll 1
              for (int i0 = 0; i0 < kKeys * kC; i0 += kIlp * kFixers) {
                uint4 x4[kIlp];
#pragma unroll
                for (int i = 0; i < kIlp; ++i) {
                  const int u = i0 + i * kFixers + ft;
                  x4[i] = u < kKeys * kC ? *reinterpret_cast<const uint4*>(raw + u * 16)
                                         : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < kIlp; ++i) {
                  const int u = i0 + i * kFixers + ft, r = u / kC, c = u % kC;
                  if (u >= kKeys * kC) break;
                  uint4 x = x4[i];
                  if (!sure) {
                    const int t = t0 + r;
                    if (t < w.lo || t >= w.len || !((got >> (r >> br_shift)) & 1u)) {
                      x = make_uint4(0u, 0u, 0u, 0u);
                    } else if (part) {
                      uint32_t* xs[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
                      for (int e = 0; e < 4; ++e) {
                        // bytes 0x7f and 0xff, NaN, become 0
                        const uint32_t nan = __vcmpeq4(*xs[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        bad |= nan != 0u;
                        *xs[e] &= ~nan;
                      }
                    }
                  }
                  const uint4 d0 = make_uint4(e4m3x2_bf16x2(x.x), e4m3x2_bf16x2(x.x >> 16),
                                              e4m3x2_bf16x2(x.y), e4m3x2_bf16x2(x.y >> 16));
                  const uint4 d1 = make_uint4(e4m3x2_bf16x2(x.z), e4m3x2_bf16x2(x.z >> 16),
                                              e4m3x2_bf16x2(x.w), e4m3x2_bf16x2(x.w >> 16));
                  uint8_t* dst = tile + (c >> 2) * P::kSpan + r * 128;
                  const int ch = (c & 3) * 2;
                  *reinterpret_cast<uint4*>(dst + ((ch ^ (r & 7)) << 4)) = d0;
                  *reinterpret_cast<uint4*>(dst + (((ch + 1) ^ (r & 7)) << 4)) = d1;
                }
              }
              if (part == 0) {
                const float* sc = reinterpret_cast<const float*>(raw + kKeys * D);
                for (int i = ft; i < 2 * kKeys; i += kFixers) {
                  const int r = i & (kKeys - 1), t = t0 + r;
                  float v = sc[i];
                  if (!sure) {
                    if (t < w.lo || t >= w.len || !((got >> (r >> br_shift)) & 1u)) {
                      v = 0.f;
                    } else if (i >= kKeys && !(fabsf(v) <= kFiniteMax)) {
                      v = 0.f;  // a value row that some must not see: as an element of V
                      bad = true;
                    }
                  }
                  scales[(nt & 3u) * 2 * kKeys + i] = v;
                }
              }
              if (bad) dirty[seq & (kDirty - 1)] = seq;
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              mbar_arrive(smem_u32(&raw_empty[rs]));
              mbar_arrive(smem_u32(&ready[s]));
            } else {
              if (part == 0) continue;  // K: scores of masked tokens are replaced
              ok = wait(&full[s], turn & 1u, quit, a.err);
              if (!ok) break;
              const uint32_t got = have[nt & 7u];
              if (cut || got != kAll >> (32 - boxes)) {
                bool bad = false;
                for (int r = ft; r < kKeys; r += kFixers) {
                  const int t = t0 + r;
                  const bool none =
                      t < w.lo || t >= w.len || !((got >> (r >> br_shift)) & 1u);
                  for (int c = 0; c < 8 * P::kHalves; ++c) {
                    // pieces in another order for every row: no bank conflicts
                    uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * P::kSpan + r * 128 +
                                                        ((((c & 7) + r) & 7) << 4));
                    if (none) {
                      *p = make_uint4(0u, 0u, 0u, 0u);
                      continue;
                    }
                    uint4 x = *p;
                    uint32_t* xs[4] = {&x.x, &x.y, &x.z, &x.w};
                    bool hit = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      if ((*xs[e] & 0x7f80u) == 0x7f80u) {
                        *xs[e] &= 0xffff0000u;
                        hit = true;
                      }
                      if ((*xs[e] & 0x7f800000u) == 0x7f800000u) {
                        *xs[e] &= 0x0000ffffu;
                        hit = true;
                      }
                    }
                    if (hit) {
                      *p = x;
                      bad = true;
                    }
                  }
                }
                if (bad) dirty[seq & (kDirty - 1)] = seq;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              }
              mbar_arrive(smem_u32(&ready[s]));
            }
          }
        }
      }
    }
  } else {
    // ============================================================== softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::kSoftmaxRegs));
    const int g = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + P::kColS(g), to = tmem + lanes + P::kColO(g),
                   tp = tmem + lanes + P::kColP(g);
    const float mul = a.scale * kLog2e;  // scores to log2 units
    const Cap cap = cap_of(a.softcap);
    // with a small cap to its y
    const float unit =
        a.softcap > 0.f ? fminf(fmaxf(mul * cap.per, -kFiniteMax), kFiniteMax) : mul;
    const int rt = r / G, rh = r - rt * G;
    const bool placed = a.window > 0 || a.slopes;  // depths matter
    uint32_t tile0 = 0;          // tiles of the CTA before the segment
    uint32_t my = 0, other = 0;  // tiles of this group, of the other
    uint32_t done[2] = {0, 0};   // segments of the groups
    uint32_t seq = 0, moved = 0;
    bool ok = true;
    for (int64_t at = begin; ok && at < end; ++seq) {
      const Segment w = segment_at(at);
      const int nk = w.k1 - w.k0, nkg = (nk + 1 - g) / 2;
      at += nk;
      const bool mine = rt < w.rows;
      const int h = w.j * G + rh;
      Sight see;
      see.rows = a.masks + int64_t(w.tok0 - w.i0) * a.words;
      see.mask = see.rows + int64_t(w.i0 + rt) * a.words;
      see.words = a.words;
      see.most = w.most;
      see.past = w.past;
      see.len = w.len;
      see.window = a.window;
      see.depth = placed && mine ? depth_of(see.mask, w.most) : 0;
      const int p = w.past + see.depth;
      see.lo = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
      if (mine && w.past + w.i0 + rt < 0) see.mask = nullptr;
      // cached tokens that this row sees; a row of no token takes whatever comes
      int rhi = 0x7fffffff, rlo = 0;
      if (mine) {
        rhi = see.mask ? w.past : 0;
        rlo = see.lo;
      }
      const float slope = GEN && a.slopes && mine ? __ldcg(a.slopes + h) * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f;
      bool holes = false;  // pages missing of a tile that the mask does not cut
      if (nkg == 0 && r == 0) mbar_arrive(smem_u32(&q_free[seq & 1u]));
      for (int i = 0; i < nkg; ++i, ++my) {
        ok = __all_sync(kAll, wait(&s_full[g], my & 1u, quit, a.err));
        if (!ok) break;
        fence_after();
        const uint32_t nt = tile0 + 2 * i + g;
        if (i + 1 == nkg && r == 0) mbar_arrive(smem_u32(&q_free[seq & 1u]));
        [[maybe_unused]] bool seen_o = false;
        const int t0 = (w.k0 + 2 * i + g) * kKeys;
        const uint32_t got = have[nt & 7u];
        const bool whole = got == kAll >> (32 - boxes);
        holes |= !whole && t0 >= w.all_lo && t0 + kKeys <= w.all_hi;
        const bool clear = __all_sync(kAll, t0 >= rlo && t0 + kKeys <= rhi) && whole;
        const float* ks = scales + ((nt & 3u) * 2) * kKeys;
        // where the tile has new tokens and depths matter: how much higher in the
        // text a key lies than in the cache
        const float* shift = shifts + (2 * g + (moved & 1u)) * kKeys;
        const bool deep = placed && t0 + kKeys > w.past;
        if (__builtin_expect(deep, 0)) {
          const int k = t0 + r - w.past;
          shifts[(2 * g + (moved & 1u)) * kKeys + r] =
              k >= 0 && k < w.most ? float(depth_of(see.rows + int64_t(k) * a.words, w.most) - k) : 0.f;
          mbar_arrive(smem_u32(&shifted[g]));
          ok = __all_sync(kAll, wait(&shifted[g], moved & 1u, quit, a.err));
          if (!ok) break;
          ++moved;
        }
        // All of the row's scores at once, and its weights at once: a TMEM access
        // takes hundreds of cycles whatever its size.
        uint32_t s[128];
        tmem_ld64<0>(ts, s);
        tmem_ld64<64>(ts + 64, s);
        wait_ld128(s);
        if constexpr (P::kOwnP) {
          fence_before();
          mbar_arrive(smem_u32(&s_read[g]));
        }
        // FP8: the key scales
        auto scaled = [&](uint32_t* x, int c) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + e);
            float f[4];
            un2(mul2(f2(x[e], x[e + 1]), f2(k.x, k.y)), f[0], f[1]);
            un2(mul2(f2(x[e + 2], x[e + 3]), f2(k.z, k.w)), f[2], f[3]);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[e + u] = __float_as_uint(f[u]);
          }
        };
        // to log2 units, the long way: the cap, the bias, a scale <= 0
        auto general = [&](uint32_t* x, int c) {
          const float base = slope * float(t0 + 32 * c - p);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(x[e]);
            if constexpr (SC == kLargeCap) {
              v = cap_large(v * mul, cap);
            } else {
              v *= unit;
              if (a.softcap > 0.f) v = cap_small(v, cap);
            }
            x[e] = __float_as_uint(v + fmaf(slope, float(e), base));
          }
          if (deep) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              x[e] = __float_as_uint(fmaf(slope, shift[32 * c + e], __uint_as_float(x[e])));
          }
        };
        auto masked = [&](uint32_t* x, int c) {
          // this row's tokens of the columns, one bit each: cached ones, new ones
          const int at0 = t0 + 32 * c;
          const int a0 = rlo - at0, a1 = rhi - at0;
          uint32_t bits = a0 <= 0 ? kAll : a0 >= 32 ? 0u : kAll << a0;
          bits &= a1 <= 0 ? 0u : a1 >= 32 ? kAll : kAll >> (32 - a1);
          const int k = at0 - w.past;  // the first column's number among the new tokens
          if (mine && see.mask && k > -32 && k < w.most) {
            uint32_t named;
            if (k < 0) {
              named = mask_word(see.mask, 0, w.most) << -k;
            } else {
              named = mask_word(see.mask, k >> 5, w.most) >> (k & 31);
              if (k & 31) named |= mask_word(see.mask, (k >> 5) + 1, w.most) << (32 - (k & 31));
            }
            if (a.window > 0) {
              for (uint32_t left = named; left; left &= left - 1u) {
                const int e = __ffs(left) - 1;
                if (see.depth - (k + e + int(shift[32 * c + e])) >= a.window) named &= ~(1u << e);
              }
            }
            bits |= named;
          }
          if (!((got >> ((32 * c) >> br_shift)) & 1u)) bits &= 0xffff0000u;
          if (!((got >> ((32 * c + 16) >> br_shift)) & 1u)) bits &= 0x0000ffffu;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((bits >> e) & 1u)) x[e] = 0xff800000u;
        };
        if constexpr (FP8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) scaled(s + 32 * c, c);
        }
        if constexpr (GEN) {
#pragma unroll
          for (int c = 0; c < 4; ++c) general(s + 32 * c, c);
        }
        if (__builtin_expect(!clear, 0)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) masked(s + 32 * c, c);
          __syncwarp();
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* x = s + 32 * c;
          mx[c] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2)
            mx[c] = max3(mx[c], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        }
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (!GEN) mt *= mul;
        if (i == 0) {
          m = mt;
        } else {
          const bool up = mt > m + 8.f;  // also from -inf, where nothing was seen yet
          if (__any_sync(kAll, up)) {
            const float f = up ? ex2(m - mt) : 1.f;
            if (up) m = mt;
            l *= f;
            // the tile before has to be in O (where the scores waited for it, it is)
            if constexpr (P::kOwnP) {
              ok = __all_sync(kAll, wait(&o_done[g], (my - 1) & 1u, quit, a.err));
              if (!ok) break;
              fence_after();
              seen_o = true;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(to + 32 * c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const uint64_t off_2 = f2(off, off);
        const uint64_t mul_2 = GEN ? f2(1.f, 1.f) : f2(mul, mul);
        uint64_t sum[2] = {0ull, 0ull};
        const float* vsc = ks + kKeys;
        uint32_t pk[64];
#pragma unroll
        for (int e = 0; e < 128; e += 4) {
          float z[4];
          un2(fma2(f2(s[e], s[e + 1]), mul_2, off_2), z[0], z[1]);
          un2(fma2(f2(s[e + 2], s[e + 3]), mul_2, off_2), z[2], z[3]);
#pragma unroll
          for (int u = 0; u < 4; ++u) z[u] = ex2(z[u]);
          sum[0] = add2(sum[0], f2(z[0], z[1]));
          sum[1] = add2(sum[1], f2(z[2], z[3]));
          if constexpr (FP8) {
            const float4 v = *reinterpret_cast<const float4*>(vsc + e);
            un2(mul2(f2(z[0], z[1]), f2(v.x, v.y)), z[0], z[1]);
            un2(mul2(f2(z[2], z[3]), f2(v.z, v.w)), z[2], z[3]);
          }
          pk[e / 2] = bf16x2(z[0], z[1]);
          pk[e / 2 + 1] = bf16x2(z[2], z[3]);
        }
        if constexpr (P::kOwnP) {  // the weights before these are read
          if (!seen_o) {
            ok = __all_sync(kAll, i == 0 || wait(&o_done[g], (my - 1) & 1u, quit, a.err));
            if (!ok) break;
            fence_after();
          }
        }
        __syncwarp();
        tmem_st64(tp, pk);
        {
          float s0, s1;
          un2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
        wait_st();
        fence_before();
        mbar_arrive(smem_u32(&p_full[g]));
      }
      if (!ok) break;

      // ---- the segment's end: both groups' maxima and sums, then their O's
      const int nko = (nk + g) / 2;  // the other group's tiles
      other += nko;
      stat[g * kRows + r] = make_float2(m, l);
      if (r == 0) misc[2 + g] = holes;
      auto o_wait = [&](int e, uint32_t tiles_of_e) {
        return wait(&o_done[e], (P::kOwnP ? tiles_of_e - 1 : done[e]) & 1u, quit, a.err);
      };
      if (nkg > 0) {
        ok = __all_sync(kAll, o_wait(g, my));
        if (!ok) break;
      }
      mbar_arrive(smem_u32(posted));
      ok = __all_sync(kAll, wait(posted, seq & 1u, quit, a.err));
      if (!ok) break;
      if (nko > 0) {
        ok = __all_sync(kAll, o_wait(1 - g, other));
        if (!ok) break;
      }
      fence_after();
      const bool two = nk > 1;
      const float2 sa = stat[r], sb = two ? stat[kRows + r] : make_float2(-INFINITY, 0.f);
      const float mm = fmaxf(sa.x, sb.x), base = mm == -INFINITY ? 0.f : mm;
      const float fa = ex2(sa.x - base), fb = ex2(sb.x - base);
      const float ll = sa.y * fa + sb.y * fb;
      const int64_t row = int64_t(w.tok0 + rt) * heads + h;
      const bool poisoned = *static_cast<volatile int*>(&dirty[(seq + 1) & (kDirty - 1)]) == int(seq + 1);
      const bool direct = w.begins && w.ends;
      float inv = 0.f;
      if (direct && mine) inv = close_row(mm, ll, a.sinks, h, g == 0 ? a.lse : nullptr, row);
      float* mypart = a.parts + (int64_t(cta) * 2 + (w.begins ? 1 : 0)) * P::kPartFloats;
#pragma unroll 1
      for (int c = g * (D / 64); c < (g + 1) * (D / 64); ++c) {
        uint32_t o[32];
        float of[32];
        __syncwarp();
        tmem_ld32(tmem + lanes + P::kColO(0) + 32 * c, o);
        wait_ld(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) of[e] = __uint_as_float(o[e]) * fa;
        if (two) {
          tmem_ld32(tmem + lanes + P::kColO(1) + 32 * c, o);
          wait_ld(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) of[e] = fmaf(__uint_as_float(o[e]), fb, of[e]);
        }
        if (mine && poisoned) {
          const uint3 x = tree_not_finite<D, FP8>(kv, see, w.b, w.j, w.k0, w.k1, w.all_lo, w.all_hi,
                                                  misc[2] || misc[3], 32 * c);
#pragma unroll
          for (int d = 0; d < 32; ++d) {
            if ((x.x >> d) & 1u) of[d] += INFINITY;
            if ((x.y >> d) & 1u) of[d] -= INFINITY;
            if ((x.z >> d) & 1u) of[d] = NAN;
          }
        }
        if (mine && direct) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(bf16x2(of[8 * e] * inv, of[8 * e + 1] * inv),
                                bf16x2(of[8 * e + 2] * inv, of[8 * e + 3] * inv),
                                bf16x2(of[8 * e + 4] * inv, of[8 * e + 5] * inv),
                                bf16x2(of[8 * e + 6] * inv, of[8 * e + 7] * inv));
        } else if (mine) {  // a part: O [D / 4][128 rows] float4, maximum [128], sum [128]
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(mypart + ((8 * c + e) * kRows + r) * 4) =
                make_float4(of[4 * e], of[4 * e + 1], of[4 * e + 2], of[4 * e + 3]);
        }
      }
      if (!direct && mine && g == 0) {
        mypart[kRows * D + r] = mm;
        mypart[kRows * (D + 1) + r] = ll;
      }
      fence_before();
      mbar_arrive(smem_u32(taken));
      ok = __all_sync(kAll, wait(taken, seq & 1u, quit, a.err));
      ++done[0];
      if (two) ++done[1];
      tile0 += nk;
    }
  }
  // ---- every role is done (or has given up): free the tensor memory
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// Joins the parts of the pieces that lie in several CTAs, launched behind the
// kernel above: a block takes eight dims of a row tile at a time, a thread a row,
// with kJoin parts' loads in flight.
constexpr int kJoinThreads = kRows;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    paged_tree_join_kernel(const KernelArgs a, int ctas, int heads) {
  constexpr int kJoin = 8;
  constexpr int kPartFloats = kRows * (D + 2);
  const int r = threadIdx.x;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int units = ctas * (D / 8);
  const int rt = r / a.group, rh = r - rt * a.group;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int cta = u / (D / 8), c = u % (D / 8);  // where the piece begins; dims 8c ..
    const int4 rec = __ldcg(a.joins + cta);        // parts, first token, tokens, kv head
    if (rt >= rec.z) continue;                     // (no parts: no tokens)
    // the first part is its CTA's second one, the others their CTAs' first ones
    auto part_at = [&](int q) {
      return a.parts + (int64_t(cta + q) * 2 + (q == 0 ? 1 : 0)) * kPartFloats;
    };
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int q0 = 0; q0 < rec.x; q0 += kJoin) {
      float4 v[kJoin][2];
      float pm[kJoin], pl[kJoin], mx = m;
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        const bool in = q0 + e < rec.x;
        const float* p = part_at(in ? q0 + e : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[e][i] = in ? __ldcg(reinterpret_cast<const float4*>(p + ((2 * c + i) * kRows + r) * 4))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        pm[e] = in ? __ldcg(p + kRows * D + r) : -INFINITY;
        pl[e] = in ? __ldcg(p + kRows * (D + 1) + r) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kJoin; ++e) mx = fmaxf(mx, pm[e]);
      const float ms = mx == -INFINITY ? 0.f : mx, old = ex2(m - ms);
      m = mx;
      l *= old;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= old;
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        const float f = ex2(pm[e] - ms);
        l = fmaf(pl[e], f, l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o[4 * i] = fmaf(v[e][i].x, f, o[4 * i]);
          o[4 * i + 1] = fmaf(v[e][i].y, f, o[4 * i + 1]);
          o[4 * i + 2] = fmaf(v[e][i].z, f, o[4 * i + 2]);
          o[4 * i + 3] = fmaf(v[e][i].w, f, o[4 * i + 3]);
        }
      }
    }
    const int h = rec.w * a.group + rh;
    const int64_t row = int64_t(rec.y + rt) * heads + h;
    const float inv = close_row(m, l, a.sinks, h, c == 0 ? a.lse : nullptr, row);
    *reinterpret_cast<uint4*>(a.out + row * D + 8 * c) =
        make_uint4(bf16x2(o[0] * inv, o[1] * inv), bf16x2(o[2] * inv, o[3] * inv),
                   bf16x2(o[4] * inv, o[5] * inv), bf16x2(o[6] * inv, o[7] * inv));
  }
}

template <int D, bool FP8, Scores SC>
cudaError_t launch_as(const DeviceInfo& di, const PagedKv& kv, const TreeArgs& t, cudaStream_t s,
                      bool pdl) {
  using P = Plan<D, FP8>;
  auto kern = paged_tree_kernel<D, FP8, SC>;
  const PagedAttnArgs& a = t.attn;
  const int G = a.heads / kv.kv_heads, TT = kRows / G;
  CUtensorMap mq, mk = {}, mv = {};
  {
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(a.heads), cuuint64_t(a.tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(a.q_stride) * 2};
    const cuuint32_t box[3] = {64u, cuuint32_t(G), cuuint32_t(TT)};
    if (cudaError_t e = encode(&mq, a.q, 3, dims, strides, box)) return e;
  }
  if (!FP8) {
    const cuuint64_t dims[2] = {cuuint64_t(D),
                                (cuuint64_t(kv.num_pages) * kv.kv_heads) << kv.page_shift};
    const cuuint64_t strides[1] = {cuuint64_t(D) * 2};
    const cuuint32_t box[2] = {64u, 1u << kv.page_shift};
    if (cudaError_t e = encode(&mk, kv.k, 2, dims, strides, box)) return e;
    if (cudaError_t e = encode(&mv, kv.v, 2, dims, strides, box)) return e;
  }
  static const bool fits = has_registers(kern, P::kLaunchRegs);
  if (!fits) return cudaErrorInvalidDeviceFunction;
  if (cudaError_t e = ensure_smem(di, kern, P::kSmem)) return e;
  const int ctas = di.sms < kMaxCtas ? di.sms : kMaxCtas;
  KernelArgs d;
  d.starts = a.starts;
  d.tokens = a.tokens;
  d.group = G;
  d.per_tile = TT;
  d.scale = a.scale;
  d.softcap = a.softcap;
  d.window = a.window;
  d.slopes = a.slopes;
  d.sinks = a.sinks;
  d.masks = t.masks;
  d.words = t.words;
  d.out = a.out;
  d.lse = a.lse;
  d.err = di.error_word;
  // pieces of one tile are never split
  const bool may_split = int64_t(kv.pages_per_seq) << kv.page_shift > kKeys;
  uint8_t* ws = static_cast<uint8_t*>(a.ws) + kCounters * 4;
  d.joins = may_split ? reinterpret_cast<int4*>(ws) : nullptr;
  d.parts = reinterpret_cast<float*>(ws + kMaxCtas * 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, kv, d)) return e;
  if (!may_split) return cudaSuccess;
  cfg.gridDim = dim3(unsigned(di.sms * 4));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the join always follows programmatically
  return cudaLaunchKernelEx(&cfg, paged_tree_join_kernel<D>, d, ctas, a.heads);
}

template <int D, bool FP8>
cudaError_t launch(const DeviceInfo& di, const PagedKv& kv, const TreeArgs& t, cudaStream_t s,
                   bool pdl) {
  if (t.attn.softcap > kCapSmall) return launch_as<D, FP8, kLargeCap>(di, kv, t, s, pdl);
  if (t.attn.softcap > 0.f || t.attn.slopes || !(t.attn.scale > 0.f))
    return launch_as<D, FP8, kGeneral>(di, kv, t, s, pdl);
  return launch_as<D, FP8, kPlain>(di, kv, t, s, pdl);
}

}  // namespace

size_t paged_tree_workspace_bytes(int head_dim) {
  // (the decode kernel's counters,) the records of the join, two parts of a row
  // tile per CTA
  const DeviceInfo* di = device_info();
  const int64_t ctas = di && di->sms < kMaxCtas ? di->sms : kMaxCtas;
  return size_t(kCounters) * 4 + kMaxCtas * 16 + size_t(ctas) * 2 * kRows * (head_dim + 2) * 4;
}

cudaError_t launch_paged_tree(const PagedKv& kv, int head_dim, bool fp8, const TreeArgs& a,
                              cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  if (head_dim == 64)
    return fp8 ? launch<64, true>(*di, kv, a, s, pdl) : launch<64, false>(*di, kv, a, s, pdl);
  return fp8 ? launch<128, true>(*di, kv, a, s, pdl) : launch<128, false>(*di, kv, a, s, pdl);
}

}  // namespace tt

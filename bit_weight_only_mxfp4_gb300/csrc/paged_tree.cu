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
//   P = 2^(S - m) as bf16 high + low parts, back to TMEM
//   O += P V    A operand P from TMEM, B operand V as it lies in the cache
//
// Split.  A piece is a row tile (floor(128 / G) tokens x G heads) of a sequence and
// kv head; it has ceil(length / 128) K / V tiles.  The tiles of all pieces form
// one line, of which each of two groups of four softmax warps a CTA takes an equal
// stretch, whatever the lengths are.  A piece that lies in several stretches is
// written in parts, joined in order by a second kernel.
//
// Inside a CTA the two groups have nothing to do with each other but that they share
// the SM: while one turns its scores into weights, or writes a piece's end, the
// other's products and copies run.  (Even and odd tiles of one stretch, joined in the
// CTA at a piece's end, left the copies idle for 5 us there.)
//   warps 0-3, 4-7  softmax of the groups, one thread a row
//   warps 8, 15     a group's products, issued by the warp in step, one elected lane
//   warps 9-12      a group's K tiles, or V tiles: asked for (TMA: one box per page
//                   and 64 dims; FP8: one bulk copy per page), and once there turned
//                   into bf16 in their place, if E4M3 codes, and made safe (below)
//   warps 13, 14    what is next of a group: pages looked up, FP8: scales
// Several warps ask for the copies because the asking bounds one: some 100 cycles a
// box.  Measured on copies alone, boxes of 2 KB from memory: one warp 2.8 TB/s, two
// 4.9, four 6.7; from L2 3.1, 6.0, 10.9.  (Copied 16 bytes a lane by cp.async, an
// instruction took 100 cycles.)
// The running maximum is only raised (and O rescaled) when a row's maximum has
// grown by more than 2^8.
//
// Measured (back to back in a graph): 8 new tokens on 332, 16 / 4 heads of 128, 16.7 us (a
// start, one or two tiles, the join); 64 on 32767, 64 / 8 heads of 64, 86.8 us (0.21 of the
// bf16 rate: S -> softmax -> P V of a row tile, 5132 warp instructions, 46% of the issue
// slots; without softmax 68); 32 ragged sequences, up
// to 16 on up to 8191, 16 / 4 heads of 128, 69.7 us (3.9 TB/s; without softmax 64.5); 48, up
// to 24 on up to 12000, 64 / 8 heads of 64 in FP8, 284 us (without conversion 259, without
// softmax 226, without both 176: four converting and eight softmax warps share the issue
// slots, 51% busy, 7543 instructions a tile).  With weights rounded once to bf16 these
// were 15.1, 59.2, 63.8 and 249; their low parts alone, left out, give 16.5, 81.1, 68.6 and
// 271 (the rest: two stores and waits for P, and its products twice).
//
// Rounding.  Q and K products are exact, sums 32-bit; P is a bf16 high and low part
// (2^-16 of each weight, as in the decode kernel: a drafted step's output should not
// lose to the step that it takes the place of); the sum of weights is taken from the
// unrounded ones.  FP8: codes become bf16 exactly, the scales multiply S and P in 32 bits.
//
// Masked values.  0 * NaN is NaN, so a V row that some row must not see (a new
// token's, or one that the window cuts) may not enter the product with NaN or
// infinities in it: those elements are zeroed, and the rows that do see them get
// them added at the end.  Rows of no token are zeroed.
#include <cmath>
#include <type_traits>

#include "paged_mma.cuh"

namespace tt {
namespace {

constexpr int kMmaWarp = 8, kCopyWarp = 9, kPlanWarp = 13, kMmaWarp2 = 15;
constexpr int kMaxCtas = 1024;
constexpr int kCounters = 1024;  // the decode kernel's, at the workspace's start: left alone
constexpr int kAhead = 4;        // tiles of a group that are planned at once
constexpr int kDirty = 8;
constexpr float kBelowOne = 0x1.fffffep-1f;  // times it a weight falls by its last bit or two

// What the warps of a group know of a tile.
struct Tile {
  int32_t row[8];    // first cache row of its pages, or -1
  uint32_t got;      // pages present, a bit each
  int16_t from, upto;  // its rows of tokens
  int16_t seen0, seen1;  // those that every row of S sees
  int32_t segment;   // 1, 2, ..
  int32_t ends;      // bit 0: first of the segment, bit 1: last
  int32_t next_token, next_head;  // of the last: where the next segment's Q is, or -1
};

template <int D, bool FP8>
struct Plan {
  static constexpr int kThreads = 512;
  // registers a thread: at launch, of the softmax warps, of the others
  static constexpr int kLaunchRegs = 128;
  static constexpr int kSoftmaxRegs = 200;
  static constexpr int kOtherRegs = 56;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs,
                "register shares");
  static constexpr int kHalves = D / 64;            // 128-byte spans of a bf16 row
  static constexpr int kSpan = kKeys * 128;         // bytes of a tile's one span
  static constexpr int kTile = kSpan * kHalves;     // a K or V tile, or a Q tile
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kRow = FP8 ? D : 2 * D;      // bytes of a cache row
  // Slots of a group's K or V: tile i of the group lies in slot i % kDepth.  A slot
  // is one warp's, and one group's, so that all wait for every phase of its barriers
  // in turn.
  static constexpr int kDepth = kSlots / 4;
  static constexpr int kOffKv = 2 * kTile;                      // (each group's Q before)
  static constexpr int kOffScale = kOffKv + kSlots * kTile;     // [2][kAhead][key, value][128]
  static constexpr int kOffDepth = kOffScale + (FP8 ? 2 * kAhead * 2 * kKeys * 4 : 0);  // [2][2][128] floats
  static constexpr int kOffTiles = kOffDepth + 4 * kKeys * 4;   // Tile [2][kAhead]
  static constexpr int kOffLine = kOffTiles + (2 * kAhead * int(sizeof(Tile)) + 7) / 8 * 8;  // int64 [batch + 1]
  static constexpr int kOffStart = kOffLine + (kPagedMaxBatch + 2) * 8;
  static constexpr int kOffCount = kOffStart + kPagedMaxBatch * 4;
  static constexpr int kOffLen = kOffCount + kPagedMaxBatch * 4;
  static constexpr int kOffBar = kOffLen + kPagedMaxBatch * 4;
  static constexpr int kSmem = 1024 + kOffBar + 768;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOffBar % 8 == 0 && kOffLine % 8 == 0, "alignment");
  // TMEM columns of the groups: S, O and P, for every kChunk tokens the high parts and
  // then the low ones.  P lies over S, and the next scores wait for P V; with 64 dims of
  // bf16 the next scores wait only until S is read, and one half of P at a time has
  // columns of its own: the second one waits for the first one's products.
  static constexpr bool kOwnP = D == 64 && !FP8;
  static constexpr int kPass = FP8 ? kKeys : kKeys / 2;  // tokens that P goes to the products with
  static constexpr int kPasses = kKeys / kPass;
  // (FP8, the batch below: 64 tokens 316 us, 32 285, 128 283)
  static constexpr int kChunk = FP8 ? 32 : 64;
  static_assert(!kOwnP || kChunk == kPass, "a wait for each pass");
  __host__ __device__ static constexpr int kColS(int g) { return 128 * g; }
  __host__ __device__ static constexpr int kColO(int g) { return 256 + D * g; }
  __host__ __device__ static constexpr int kColP(int g, int pass) {
    return kOwnP ? 384 + 64 * g : kColS(g) + kPass * pass;
  }
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
  int4* joins;   // a record for each group whose last piece goes on in the next one's
  float* parts;  // [group][2]: of a piece that began before, of one that goes on
  int32_t* err;
};

// A group's part of a piece: K / V tiles [k0, k1) of the row tile that begins at
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
// each) among the tokens of [t0, t1) that the row sees and that were kept out of
// the product: those that not every row sees.
template <int D, bool FP8>
__device__ __noinline__ uint3 tree_not_finite(const PagedKv& kv, const Sight& s, int b, int j, int t0,
                                              int t1, int all_lo, int all_hi, int d0) {
  uint3 x = make_uint3(0u, 0u, 0u);
  for (int t = t0; t < t1; ++t) {
    if (t >= all_lo && t < all_hi) {
      t = all_hi - 1;
      continue;
    }
    if (!s.sees(t)) continue;
    const int page = paged_page(kv, b, t, nullptr);
    if (page < 0) continue;
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
  return x;
}

// Four E4M3 codes -> two bf16x2, exact (NaN becomes 480): with exponent and mantissa
// moved to bf16's places a code is its value times 2^-120, subnormal ones too.
// (Conversion instructions, three for two codes, share the unit with the softmax
// warps' exponentials.)
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  auto half = [](uint32_t t) {
    const uint32_t u = ((t >> 4) & 0x07f007f0u) | (t & 0x80008000u);
    const uint32_t up = 0x7b807b80u;  // 2^120
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                     *reinterpret_cast<const __nv_bfloat162*>(&up));
    return *reinterpret_cast<const uint32_t*>(&y);
  };
  lo = half(__byte_perm(w, 0u, 0x1404));
  hi = half(__byte_perm(w, 0u, 0x3424));
}

// What few K and V tiles need, by a whole warp; all are bf16 here.  V: rows of no token
// become zeros, and elements that are not finite in rows that not every row of S sees
// (true: some were).  E4M3 codes of NaN, `nan`, are 480 so far, which no other is.
template <int D, bool FP8>
__device__ __noinline__ bool tree_make_safe(uint8_t* tile, const Tile* d, int value, bool nan,
                                            int page_shift) {
  constexpr int kPieces = D / 8, kStep = 32 / kPieces;  // 16-byte pieces of a row; rows at once
  const int lane = threadIdx.x & 31, c = lane % kPieces, r0 = lane / kPieces;
  const int from = d->from, upto = d->upto, seen0 = d->seen0, seen1 = d->seen1;
  const uint32_t got = d->got;
  uint8_t* column = tile + (c >> 3) * kKeys * 128;
  auto piece = [&](int r) {
    return reinterpret_cast<uint4*>(column + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
  bool bad = false;
  auto scan = [&](int r, int end, bool hidden) {
    for (r += r0; r < end; r += kStep) {
      uint4 x = *piece(r);
      auto fixed = [&](uint32_t h) {  // one element
        if (FP8 ? (h & 0x7fffu) != 0x43f0u : (h & 0x7f80u) != 0x7f80u) return h;
        bad |= hidden;
        return hidden ? 0u : 0x7fc0u;
      };
      auto both = [&](uint32_t w) { return fixed(w & 0xffffu) | fixed(w >> 16) << 16; };
      *piece(r) = make_uint4(both(x.x), both(x.y), both(x.z), both(x.w));
    }
  };
  if (!value) {
    scan(from, upto, false);
    return false;
  }
  auto clear = [&](int r, int end) {
#pragma unroll 4
    for (r += r0; r < end; r += kStep) *piece(r) = make_uint4(0u, 0u, 0u, 0u);
  };
  clear(0, from);
  clear(upto, kKeys);
  for (int t = from; t < upto; t = ((t >> page_shift) + 1) << page_shift)
    if (!((got >> (t >> page_shift)) & 1u)) clear(t, min(((t >> page_shift) + 1) << page_shift, upto));
  __syncwarp();
  if (FP8 && !nan) return false;
  if (seen0 > from) scan(from, min(seen0, upto), true);
  if (FP8) scan(max(from, seen0), min(seen1, upto), false);
  if (seen1 < upto) scan(max(seen1, from), upto, true);
  return bad;
}

// A chunk of P to its columns (complete after wait_st).
__device__ __forceinline__ void tmem_put(uint32_t addr, const uint32_t (&r)[32]) { tmem_st32(addr, r); }
__device__ __forceinline__ void tmem_put(uint32_t addr, const uint32_t (&r)[64]) { tmem_st64(addr, r); }

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
  constexpr int kThreads = P::kThreads;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + P::kOffScale);
  float* shifts = reinterpret_cast<float*>(smem + P::kOffDepth);
  Tile* plans = reinterpret_cast<Tile*>(smem + P::kOffTiles);  // [group][kAhead]
  int64_t* line = reinterpret_cast<int64_t*>(smem + P::kOffLine);  // tiles before a sequence's
  int32_t* first = reinterpret_cast<int32_t*>(smem + P::kOffStart);
  int32_t* count = reinterpret_cast<int32_t*>(smem + P::kOffCount);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + P::kOffLen);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kOffBar);  // of the slots
  uint64_t* empty = full + P::kSlots;
  uint64_t* ready = empty + P::kSlots;   // made safe, or converted
  uint64_t* planned = ready + P::kSlots;  // [2][kAhead]
  uint64_t* freed = planned + 2 * kAhead;   // [2][kAhead], when a tile is used up
  uint64_t* q_full = freed + 2 * kAhead;    // [2], of the groups, and so on
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;  // [pass][2]
  uint64_t* o_done = p_full + 4;
  uint64_t* half_done = o_done + 2;
  uint64_t* s_read = half_done + 2;
  uint64_t* shifted = s_read + 2;
  uint64_t* drained = shifted + 2;
  int* dirty = reinterpret_cast<int*>(drained + 2);  // [2][kDirty] segment
  int* misc = dirty + 2 * kDirty;  // [0] TMEM address, [1] quit
  volatile int* quit = misc + 1;
  int64_t* scan = reinterpret_cast<int64_t*>(smem);  // [warps], before the main loop

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P::kSlots; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
      mbar_init(smem_u32(&ready[i]), 1);
    }
    for (int i = 0; i < 2 * kAhead; ++i) {
      mbar_init(smem_u32(&planned[i]), 1);
      mbar_init(smem_u32(&freed[i]), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&q_full[g]), 1);
      mbar_init(smem_u32(&s_full[g]), 1);
      mbar_init(smem_u32(&p_full[g]), kRows);
      mbar_init(smem_u32(&p_full[2 + g]), kRows);
      mbar_init(smem_u32(&o_done[g]), 1);
      mbar_init(smem_u32(&half_done[g]), 1);
      mbar_init(smem_u32(&s_read[g]), kRows);
      mbar_init(smem_u32(&shifted[g]), kRows);
      mbar_init(smem_u32(&drained[g]), 1);
    }
    for (int i = 0; i < 2 * kDirty; ++i) dirty[i] = 0;
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
  // The groups' stretches of the line: equal shares of it, two tiles at least.
  const int64_t total = line[kv.batch];
  const int all = 2 * gridDim.x, own = 2 * blockIdx.x;  // groups, this CTA's first one
  const int groups = total >= 2 * all ? all : int((total + 1) / 2);
  auto stretch = [&](int i) { return i < groups ? total * i / groups : total; };
  const int64_t begins[2] = {stretch(own), stretch(own + 1)}, ends[2] = {begins[1], stretch(own + 2)};

  // A walk over a group's segments: at a piece (its number in the sequence) and a
  // tile of it; `left` tiles of the stretch.
  struct Walk {
    int64_t left;
    int b, piece, tile, tiles, pieces;
  };
  auto walk_to = [&](int64_t at, int64_t end) {
    Walk k;
    k.left = end - at;
    if (k.left <= 0) return k;
    int lo = 0, hi = kv.batch;  // the last b with line[b] <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (line[mid] <= at) lo = mid; else hi = mid;
    }
    k.b = lo;
    k.tiles = tiles_of(lo);
    k.pieces = row_tiles(lo) * kv.kv_heads;
    const int64_t rem = at - line[lo];
    k.piece = rem >> 31 ? int(rem / k.tiles) : int(uint32_t(rem) / uint32_t(k.tiles));
    k.tile = int(rem - int64_t(k.piece) * k.tiles);
    return k;
  };
  auto next_segment = [&](Walk& k) {
    Segment w;
    const int b = k.b, rts = row_tiles(b), n = count[b];
    w.b = b;
    w.j = k.piece / rts;
    w.i0 = (k.piece - w.j * rts) * TT;
    w.tok0 = first[b] + w.i0;
    w.rows = n - w.i0 < TT ? n - w.i0 : TT;
    w.len = lens[b];
    w.past = w.len - n;
    w.most = n < 32 * a.words ? n : 32 * a.words;
    w.lo = low_of(w.past);
    w.all_hi = w.past > 0 ? w.past : 0;
    // the deepest row's window
    w.all_lo = a.window > 0 && w.past + w.most > a.window ? w.past + w.most - a.window : 0;
    w.begins = k.tile == 0;
    w.ends = k.left >= k.tiles - k.tile;
    const int nk = w.ends ? k.tiles - k.tile : int(k.left);
    w.k0 = w.lo / kKeys + k.tile;
    w.k1 = w.k0 + nk;
    k.left -= nk;
    k.tile = 0;
    if (++k.piece == k.pieces && k.left > 0) {
      do ++k.b; while (line[k.b + 1] == line[k.b]);
      k.piece = 0;
      k.tiles = tiles_of(k.b);
      k.pieces = row_tiles(k.b) * kv.kv_heads;
    }
    return w;
  };
  // the record of the piece that begins in a group's stretch and goes on in the next
  if (tid < 2 && a.joins) {
    int4 rec = make_int4(0, 0, 0, 0);
    const int64_t begin = begins[tid], end = ends[tid];
    if (end > begin) {
      const Walk k = walk_to(end - 1, end);
      const int64_t from = end - 1 - k.tile;
      if (from >= begin && from + k.tiles > end) {
        const int last = int(((from + k.tiles) * groups + total - 1) / total) - 1;
        const int rts = row_tiles(k.b), i0 = (k.piece % rts) * TT, n = count[k.b] - i0;
        rec = make_int4(last - (own + tid) + 1, first[k.b] + i0, n < TT ? n : TT, k.piece / rts);
      }
    }
    a.joins[own + tid] = rec;
  }
  const int boxes = kKeys >> kv.page_shift;  // pages of a tile

  // A group's Q, rows of TT tokens from a token on, of a kv head.
  auto load_q = [&](int g, int token, int j) {
    const uint32_t bar = smem_u32(&q_full[g]);
    mbar_arrive_expect_tx(bar, uint32_t(TT * G * 128 * P::kHalves));
    for (int h = 0; h < P::kHalves; ++h)
      tma_q(sbase + g * P::kTile + h * P::kSpan, &map_q, 64 * h, j * G, token, bar);
  };

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kOtherRegs));
    const int64_t tiles_all[2] = {ends[0] - begins[0], ends[1] - begins[1]};
    // the slot of a group's tile i, K or V
    auto slot_of = [](int g, int value, uint32_t i) {
      return ((i % P::kDepth) * 2 + g) * 2 + value;
    };
    const int in_page = (1 << kv.page_shift) - 1;
    if (warp >= kPlanWarp && warp < kPlanWarp + 2) {
      // ============================================================== plans
      // A lane a page, then (FP8) four tokens a lane.  A tile's entries are asked for
      // two tiles ahead, its scales one; it is planned when the one kAhead before it is
      // used up: its places in the rings are free then.
      const int g = warp - kPlanWarp;
      Walk walk = walk_to(begins[g], ends[g]);
      struct Next {  // a tile: what is needed of its segment
        int b, j, kt, k0, k1, lo, len, all_lo, all_hi, segment;
      };
      Next u;
      u.segment = 0;
      u.kt = u.k1 = 0;
      int token = -1;
      // goes on to the next tile; false at the end
      auto advance = [&] {
        if (++u.kt < u.k1) return true;
        if (walk.left <= 0) return false;
        const Segment w = next_segment(walk);
        u = {w.b, w.j, w.k0, w.k0, w.k1, w.lo, w.len, w.all_lo, w.all_hi, u.segment + 1};
        token = w.tok0;
        return true;
      };
      auto look = [&] {  // the table's entry of this lane's page
        const int t = u.kt * kKeys + (lane << kv.page_shift);
        const bool in = lane < boxes && t < u.len && t + (1 << kv.page_shift) > u.lo;
        return in ? __ldcg(kv.page_table + int64_t(u.b) * kv.pages_per_seq + (t >> kv.page_shift))
                  : -1;
      };
      float v[2][kKeys / 32];
      auto load_scales = [&](const Next& n, int row0) {
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) {
            const int r = 32 * i + lane, t = n.kt * kKeys + r;
            const int first_row = __shfl_sync(kAll, row0, r >> kv.page_shift);
            const bool some = first_row >= 0 && t >= n.lo && t < n.len;
            v[0][i] = some ? __ldcg(kv.k_scales + first_row + (r & in_page)) : 0.f;
            v[1][i] = some ? __ldcg(kv.v_scales + first_row + (r & in_page)) : 0.f;
          }
        }
      };
      auto row_of = [&](int entry, int j) {
        if (entry >= kv.num_pages) {
          flag_error(a.err, kErrShape);
          entry = -1;
        }
        return entry >= 0 ? (entry * kv.kv_heads + j) << kv.page_shift : -1;
      };
      bool more = advance();
      if (more) {
        if (lane == 0) load_q(g, token, u.j);
        Next now = u;
        int row = row_of(look(), u.j);
        load_scales(now, row);
        more = advance();
        int entry = more ? look() : -1;
        for (uint32_t i = 0;; ++i) {
          const uint32_t ring = i % kAhead;
          if (i >= kAhead &&
              !__all_sync(kAll, wait(&freed[g * kAhead + ring], (i / kAhead - 1u) & 1u, quit, a.err)))
            break;
          const uint32_t got = __ballot_sync(kAll, row >= 0);
          const int t0 = now.kt * kKeys;
          auto within = [&](int t) { return int16_t(t < t0 ? 0 : t - t0 > kKeys ? kKeys : t - t0); };
          Tile* d = plans + g * kAhead + ring;
          if (lane < 8) d->row[lane] = row;
          if (lane == 0) {
            const bool last = now.kt + 1 == now.k1;
            d->got = got;
            d->from = within(now.lo);
            d->upto = within(now.len);
            d->seen0 = within(now.all_lo);
            d->seen1 = within(now.all_hi);
            d->segment = now.segment;
            d->ends = (now.kt == now.k0 ? 1 : 0) | (last ? 2 : 0);
            d->next_token = last && more ? token : -1;
            d->next_head = u.j;
          }
          if constexpr (FP8) {
            float* to = scales + (g * kAhead + ring) * 2 * kKeys;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < kKeys / 32; ++e) {
              const int r = 32 * e + lane, t = t0 + r;
              // a value row's scale, as an element of V
              if ((t < now.all_lo || t >= now.all_hi) && !(fabsf(v[1][e]) <= kFiniteMax)) {
                v[1][e] = 0.f;
                bad = true;
              }
              to[r] = v[0][e];
              to[kKeys + r] = v[1][e];
            }
            if (bad) dirty[g * kDirty + now.segment % kDirty] = now.segment;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&planned[g * kAhead + ring]));
          if (!more) break;
          now = u;
          row = row_of(entry, u.j);
          load_scales(now, row);
          more = advance();
          if (more) entry = look();
        }
      }
    } else if (warp >= kCopyWarp && warp < kPlanWarp) {
      // ============================================================ copies
      const int g = (warp - kCopyWarp) >> 1, value = (warp - kCopyWarp) & 1;
      const uint32_t parts = uint32_t(tiles_all[g]);
      // E4M3 codes are copied into their slot's last bytes (64 dims), or second span
      // (128)
      constexpr uint32_t kRaw = FP8 ? P::kTile / 2 : 0;
      constexpr int kPieces = P::kRow / 16, kStep = 32 / kPieces;  // rows for 32 lanes
      const int c = lane % kPieces, r0 = lane / kPieces;
      const uint32_t whole = kAll >> (32 - boxes);
      // Whether part i may be asked for: its tile is planned, its slot is free.
      auto may_ask = [&](uint32_t i, bool block) {
        uint64_t* p = &planned[g * kAhead + i % kAhead];
        uint64_t* e = &empty[slot_of(g, value, i)];
        const uint32_t pp = (i / kAhead) & 1u, ep = (i / P::kDepth - 1u) & 1u;
        bool go;
        if (block)
          go = wait(p, pp, quit, a.err) && (i < P::kDepth || wait(e, ep, quit, a.err));
        else
          go = mbar_test_wait(smem_u32(p), pp) && (i < P::kDepth || mbar_test_wait(smem_u32(e), ep));
        return bool(__all_sync(kAll, go));
      };
      auto ask = [&](uint32_t i) {
        const Tile* d = plans + g * kAhead + i % kAhead;
        const uint32_t s = slot_of(g, value, i), bar = smem_u32(&full[s]);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, __popc(d->got) * (uint32_t(P::kRow) << kv.page_shift));
        __syncwarp();
        const int row = lane < boxes ? d->row[lane] : -1;
        const uint32_t dst = sbase + P::kOffKv + s * P::kTile + kRaw;
        if (row >= 0) {
          if constexpr (FP8) {
            const uint8_t* pool = static_cast<const uint8_t*>(value ? kv.v : kv.k);
            bulk_copy(dst + ((uint32_t(lane) * P::kRow) << kv.page_shift),
                      pool + int64_t(row) * P::kRow, uint32_t(P::kRow) << kv.page_shift, bar);
          } else {
            for (int h = 0; h < P::kHalves; ++h)
              tma_rows(dst + (uint32_t(lane) << (kv.page_shift + 7)) + h * P::kSpan,
                       value ? &map_v : &map_k, 64 * h, row, bar);
          }
        }
        __syncwarp();
      };
      // A part that has landed is turned into bf16, made safe, handed to the tensor
      // cores.  E4M3 codes: in place, in rising order of rows: a row's bf16 elements
      // end before the codes of the next ones begin, or lie where its own were.  (What
      // few tiles need is a function of its own: in the loop it cost 80 us of 320, 48
      // ragged sequences of 64 / 8 heads of 64.)
      constexpr int kIlp = 4;
      constexpr int kSteps = FP8 ? kKeys / (kStep * kIlp) : 1;
      uint32_t odd = 0u;  // carries into the top bits of bytes from 0x7f and 0xff, NaN
      bool bad = false;
      auto work = [&](uint32_t n, int step) {
        uint8_t* tile = smem + P::kOffKv + slot_of(g, value, n) * P::kTile;
        if constexpr (FP8) {
          uint4 x[kIlp];
#pragma unroll
          for (int i = 0; i < kIlp; ++i)
            x[i] = *reinterpret_cast<const uint4*>(
                tile + kRaw + ((step * kIlp + i) * kStep + r0) * P::kRow + 16 * c);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kIlp; ++i) {
            const int r = (step * kIlp + i) * kStep + r0;
            odd |= ((x[i].x & 0x7f7f7f7fu) + 0x01010101u) | ((x[i].y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((x[i].z & 0x7f7f7f7fu) + 0x01010101u) | ((x[i].w & 0x7f7f7f7fu) + 0x01010101u);
            uint4 d0, d1;
            e4m3x4_bf16(x[i].x, d0.x, d0.y);
            e4m3x4_bf16(x[i].y, d0.z, d0.w);
            e4m3x4_bf16(x[i].z, d1.x, d1.y);
            e4m3x4_bf16(x[i].w, d1.z, d1.w);
            uint8_t* dst = tile + (c >> 2) * P::kSpan + r * 128;
            const int ch = (c & 3) * 2;
            *reinterpret_cast<uint4*>(dst + ((ch ^ (r & 7)) << 4)) = d0;
            *reinterpret_cast<uint4*>(dst + (((ch + 1) ^ (r & 7)) << 4)) = d1;
          }
          __syncwarp();
        }
        if (step + 1 == kSteps) {
          const Tile* d = plans + g * kAhead + n % kAhead;
          const bool edge = d->from > 0 || d->upto < kKeys || d->got != whole;
          const bool cut = d->seen0 > d->from || d->seen1 < d->upto;
          const bool nan = FP8 && __any_sync(kAll, (odd & 0x80808080u) != 0u);
          if (nan || (value && (edge || (!FP8 && cut)))) {
            bad = tree_make_safe<D, FP8>(tile, d, value, nan, kv.page_shift);
            __syncwarp();
          }
          odd = 0u;
        }
      };
      auto hand_over = [&](uint32_t n) {
        const Tile* d = plans + g * kAhead + n % kAhead;
        if (bad) dirty[g * kDirty + d->segment % kDirty] = d->segment;
        bad = false;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ready[slot_of(g, value, n)]));
      };
      uint32_t asked = 0, done = 0;
      if (!FP8 && !value) {  // bf16 keys need nothing: scores of masked tokens are replaced
        for (; asked < parts && may_ask(asked, true); ++asked) ask(asked);
      } else {
        for (int step = 0; done < parts;) {
          // as many parts on their way as there are slots; it is waited for one only where
          // nothing else is left to do
          while (asked < parts && asked - done < P::kDepth && may_ask(asked, false)) ask(asked++);
          if (asked == done) {
            if (!may_ask(asked, true)) break;
            continue;
          }
          if (step == 0 && !__all_sync(kAll, wait(&full[slot_of(g, value, done)],
                                                   (done / P::kDepth) & 1u, quit, a.err)))
            break;
          work(done, step);
          if (++step < kSteps) continue;
          step = 0;
          hand_over(done++);
        }
      }
      // nothing lands after the CTA's end (where the warp gave up)
      for (uint32_t i = 1; i <= P::kDepth && i <= asked; ++i)
        (void)mbar_wait_bounded(smem_u32(&full[slot_of(g, value, asked - i)]),
                                ((asked - i) / P::kDepth) & 1u);
    } else {
      // ========================================================== products
      // A warp for each group, issued by the warp in step.  (One for both took 2700
      // cycles for a round of both groups' products: 75.9 us for 64.3, one sequence of 32768
      // tokens, 64 new ones of 64 / 8 heads of 64.)  The commits free the slots, so
      // that a copy begins as soon as the products are through with its place.  Products
      // finish in order, so scores that are there say that the P V issued before them is
      // done.
      // (asked for by a vote, so that the compiler knows it to be the same in all lanes)
      const uint32_t g = __any_sync(kAll, warp == kMmaWarp2) ? 1 : 0;
      const uint32_t kv0 = sbase + P::kOffKv;
      bool ok = tmem == 0;  // all columns are ours, so they begin at 0
      if (!ok && lane == 0) {
        *quit = 1;
        flag_error(a.err, kErrShape);
      }
      // (Loops that are not unrolled: the instructions of all roles have to fit the caches.  Unrolled, 78 us for 68, 32 ragged sequences
      // of 16 / 4 heads of 128.)
      auto scores = [&](uint32_t i) {
        const uint32_t slot = slot_of(g, 0, i);
        const uint64_t q = desc_k(sbase + g * P::kTile), k = desc_k(kv0 + slot * P::kTile);
#pragma unroll 1
        for (int e = 0; e < D / 16; ++e) {
          const uint64_t off = ((e >> 2) * P::kSpan + (e & 3) * 32) >> 4;
          mma_ss(P::kColS(g), q + off, k + off, idesc(kKeys, false), e > 0);
        }
        commit(smem_u32(&s_full[g]));
        commit(smem_u32(&empty[slot]));
      };
      auto values = [&](uint32_t i, int pass, int ends) {
        const uint32_t slot = slot_of(g, 1, i);
        const uint64_t v = desc_mn(kv0 + slot * P::kTile, P::kHalves > 1 ? P::kSpan : 1024);
#pragma unroll 1
        for (int k = 0; k < 2 * P::kPass / 16; ++k) {  // (16 tokens' high or low parts)
          constexpr int kIn = P::kChunk / 16;
          const int at = pass * (P::kPass / 16) + k / (2 * kIn) * kIn + k % kIn;
          mma_ts(P::kColO(g), P::kColP(g, pass) + 8 * k, v + at * (2048 >> 4), idesc(D, true),
                 pass + k > 0 ? 1u : uint32_t(!(ends & 1)));
        }
        if (pass + 1 < P::kPasses) {
          if (P::kOwnP) commit(smem_u32(&half_done[g]));
        } else {
          commit(smem_u32(&empty[slot]));
          if (P::kOwnP || __any_sync(kAll, ends & 2)) commit(smem_u32(&o_done[g]));
        }
      };
      // Tiles, P V issued, scores issued, segments whose scores are all issued.  Where P has
      // its own columns a tile's scores go out before the P V of the tile before, unless a
      // new segment begins with it, whose Q may be late; where P lies over S, P V goes first.
      const uint32_t n = uint32_t(tiles_all[g]);
      uint32_t v = 0, sc = 0, seg = 0;
      auto await = [&](uint64_t* bar, uint32_t phase) {
        ok = ok && __all_sync(kAll, wait(bar, phase & 1u, quit, a.err));
      };
      while (ok && v < n) {
        const bool ahead = P::kOwnP && sc == v + 1 && !(plans[g * kAhead + v % kAhead].ends & 2);
        if (__any_sync(kAll, sc < n && (sc == v || ahead))) {
          await((FP8 ? ready : full) + slot_of(g, 0, sc), sc / P::kDepth);
          if (P::kOwnP) await(&s_read[g], sc - 1u);
          await(&q_full[g], seg);
          if (!ok) break;
          fence_after();
          const int ends = plans[g * kAhead + sc % kAhead].ends;
          scores(sc++);
          seg += (ends >> 1) & 1;
        } else {
          await(&ready[slot_of(g, 1, v)], v / P::kDepth);
          const int ends = plans[g * kAhead + v % kAhead].ends;
#pragma unroll 1
          for (int pass = 0; pass < P::kPasses; ++pass) {
            await(&p_full[2 * pass + g], v);
            if (!ok) break;
            fence_after();
            values(v, pass, ends);
          }
          ++v;
        }
      }
      // nothing of the tensor cores is under way when the CTA ends
      commit(smem_u32(&drained[g]));
      (void)mbar_wait_bounded(smem_u32(&drained[g]), 0);
      __syncwarp();
    }
  } else {
    // ============================================================== softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::kSoftmaxRegs));
    const int g = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + P::kColS(g), to = tmem + lanes + P::kColO(g);
    const float mul = a.scale * kLog2e;  // scores to log2 units
    const Cap cap = cap_of(a.softcap);
    // with a small cap to its y
    const float unit =
        a.softcap > 0.f ? fminf(fmaxf(mul * cap.per, -kFiniteMax), kFiniteMax) : mul;
    const int rt = r / G, rh = r - rt * G;
    const bool placed = a.window > 0 || a.slopes;  // depths matter
    uint32_t my = 0, seq = 0, moved = 0;  // tiles; segments; tiles where depths mattered
    uint32_t asked = 1;  // Q tiles
    bool ok = true;
    for (Walk walk = walk_to(begins[g], ends[g]); ok && walk.left > 0; ++seq) {
      const Segment w = next_segment(walk);
      const int nk = w.k1 - w.k0;
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
      for (int i = 0; i < nk; ++i, ++my) {
        ok = __all_sync(kAll, wait(&s_full[g], my & 1u, quit, a.err));
        if (!ok) break;
        fence_after();
        [[maybe_unused]] bool seen_o = false;
        const int t0 = (w.k0 + i) * kKeys;
        const uint32_t ring = g * kAhead + my % kAhead;
        const uint32_t got = plans[ring].got;
        // the P V issued before these scores are done
        if (!P::kOwnP && i > 0 && r == 0) mbar_arrive(smem_u32(&freed[g * kAhead + (my - 1) % kAhead]));
        // Q is done with when the segment's last scores are there
        if (r == 0 && i + 1 == nk && plans[ring].next_token >= 0) {
          load_q(g, plans[ring].next_token, plans[ring].next_head);
          ++asked;
        }
        const bool whole = got == kAll >> (32 - boxes);
        const bool clear = __all_sync(kAll, t0 >= rlo && t0 + kKeys <= rhi) && whole;
        const float* ks = scales + ring * 2 * kKeys;
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
          if (!((got >> ((32 * c) >> kv.page_shift)) & 1u)) bits &= 0xffff0000u;
          if (!((got >> ((32 * c + 16) >> kv.page_shift)) & 1u)) bits &= 0x0000ffffu;
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
        // The weights as high + low bf16 parts.  Over a bf16 cache the high one is cut off
        // below the weight, so that the low one is above 0 and both take an infinite value to
        // the same infinity (0 * infinity is NaN); an FP8 cache has none, and its weights
        // times scales may be below 0.
        constexpr int kChunk = P::kChunk;
        uint32_t pk[kChunk];  // high parts, low parts
        auto split = [&](int at, float x, float y) {
          const uint64_t z = f2(x, y);
          float a, b;
          un2(FP8 ? z : mul2(z, f2(kBelowOne, kBelowOne)), a, b);
          const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
          pk[at] = __byte_perm(ha, hb, 0x7632);
          un2(fma2(f2(ha, hb), f2(-1.f, -1.f), z), a, b);
          pk[kChunk / 2 + at] = bf16x2(a, b);
        };
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
          split(e % kChunk / 2, z[0], z[1]);
          split(e % kChunk / 2 + 1, z[2], z[3]);
          if ((e + 4) % kChunk != 0) continue;
          if constexpr (P::kOwnP) {  // the weights before these are read
            if (e >= P::kPass) {
              ok = __all_sync(kAll, wait(&half_done[g], my & 1u, quit, a.err));
            } else {
              ok = __all_sync(kAll, i == 0 || seen_o || wait(&o_done[g], (my - 1) & 1u, quit, a.err));
              if (ok && i > 0 && r == 0) mbar_arrive(smem_u32(&freed[g * kAhead + (my - 1) % kAhead]));
            }
            if (!ok) break;
            fence_after();
          }
          __syncwarp();
          tmem_put(tmem + lanes + P::kColP(g, e / P::kPass) + e % P::kPass / kChunk * kChunk, pk);
          if ((e + 4) % P::kPass == 0) {
            wait_st();
            fence_before();
            mbar_arrive(smem_u32(&p_full[e / P::kPass * 2 + g]));
          }
        }
        if (!ok) break;
        {
          float s0, s1;
          un2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
      }
      if (!ok) break;

      // ---- the segment's end
      ok = __all_sync(kAll, wait(&o_done[g], (P::kOwnP ? my - 1 : seq) & 1u, quit, a.err));
      if (!ok) break;
      fence_after();
      if (r == 0) mbar_arrive(smem_u32(&freed[g * kAhead + (my - 1) % kAhead]));
      const int64_t row = int64_t(w.tok0 + rt) * heads + h;
      const bool poisoned =
          *static_cast<volatile int*>(&dirty[g * kDirty + (seq + 1) % kDirty]) == int(seq + 1);
      const bool direct = w.begins && w.ends;
      float inv = 0.f;
      if (direct && mine) inv = close_row(m, l, a.sinks, h, a.lse, row);
      float* mypart = a.parts + (int64_t(own + g) * 2 + (w.begins ? 1 : 0)) * P::kPartFloats;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        float of[32];
        __syncwarp();
        tmem_ld32(to + 32 * c, o);
        wait_ld(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) of[e] = __uint_as_float(o[e]);
        if (mine && poisoned) {
          const uint3 x =
              tree_not_finite<D, FP8>(kv, see, w.b, w.j, max(w.k0 * kKeys, w.lo),
                                      min(w.k1 * kKeys, w.len), w.all_lo, w.all_hi, 32 * c);
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
      if (!direct && mine) {
        mypart[kRows * D + r] = m;
        mypart[kRows * (D + 1) + r] = l;
      }
      fence_before();
    }
    // no copy of Q is under way when the CTA ends
    if (r == 0 && begins[g] < ends[g]) (void)mbar_wait_bounded(smem_u32(&q_full[g]), (asked - 1) & 1u);
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
    paged_tree_join_kernel(const KernelArgs a, int groups, int heads) {
  constexpr int kJoin = 8;
  constexpr int kPartFloats = kRows * (D + 2);
  const int r = threadIdx.x;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int units = groups * (D / 8);
  const int rt = r / a.group, rh = r - rt * a.group;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int from = u / (D / 8), c = u % (D / 8);  // where the piece begins; dims 8c ..
    const int4 rec = __ldcg(a.joins + from);        // parts, first token, tokens, kv head
    if (rt >= rec.z) continue;                      // (no parts: no tokens)
    // the first part is its group's second one, the others their groups' first ones
    auto part_at = [&](int q) {
      return a.parts + (int64_t(from + q) * 2 + (q == 0 ? 1 : 0)) * kPartFloats;
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
  d.parts = reinterpret_cast<float*>(ws + 2 * kMaxCtas * 16);
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
  cfg.gridDim = dim3(unsigned(di.sms * 8));  // (4 an SM: 65 us for 59.6, the long context)
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the join always follows programmatically
  return cudaLaunchKernelEx(&cfg, paged_tree_join_kernel<D>, d, 2 * ctas, a.heads);
}

template <int D, bool FP8>
cudaError_t launch(const DeviceInfo& di, const PagedKv& kv, const TreeArgs& t, cudaStream_t s,
                   bool pdl) {
  // A kernel for each, since all of it is done for every score.  The three batches and
  // contexts above (32 ragged / FP8 / one long): plain 69.5 / 284 / 86.8 us, in the general
  // kernel 100 / 384 / 132; a cap of 30 in that one 122 / 510 / 171, in the one for large
  // caps 178 / 768 / 246; a bias 105 / 400 / 137.
  if (t.attn.softcap > kCapSmall) return launch_as<D, FP8, kLargeCap>(di, kv, t, s, pdl);
  if (t.attn.softcap > 0.f || t.attn.slopes || !(t.attn.scale > 0.f))
    return launch_as<D, FP8, kGeneral>(di, kv, t, s, pdl);
  return launch_as<D, FP8, kPlain>(di, kv, t, s, pdl);
}

}  // namespace

size_t paged_tree_workspace_bytes(int head_dim) {
  // (the decode kernel's counters,) the records of the join, two parts of a row
  // tile per group
  const DeviceInfo* di = device_info();
  const int64_t ctas = di && di->sms < kMaxCtas ? di->sms : kMaxCtas;
  return size_t(kCounters) * 4 + 2 * kMaxCtas * 16 +
         size_t(ctas) * 4 * kRows * (head_dim + 2) * 4;
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

// Attention of several new tokens per sequence over the paged cache: the
// attention of a prompt, or of a chunk of one.
//
//   z[r][t] = f(scale * q[r] . k[j][t]) + slope[h] * (t - p)
//   out[r]  = sum_t e^z v[j][t] / (sum_t e^z + e^sink[h])
//
// A row r is one new token (place p) and one of the G query heads of kv head
// j; it sees the tokens [rlo, rhi): rhi = max(p + 1, prefix) up to the length,
// rlo = p + 1 - window.  The work is 4 head_dim operations per row and
// token, so it belongs to the tensor cores:
//   S = Q K^T   128 rows x 128 tokens, tcgen05.mma, accumulator in TMEM
//   P = 2^(S - m) in bf16, back to TMEM: over S, or with 64 dims, where columns
//                 are left, into its own, so that the next S need not wait for P V
//   O += P V    A operand P from TMEM, B operand V as it lies in the cache
//               (token rows: the "transposed" B of the instruction), O in TMEM
//
// Tiles.  A row tile packs floor(128 / G) tokens x G heads, so a K and V tile
// serves the whole group and short chunks still fill rows.  A CTA works on
// two row tiles at once (A and B), each with a warpgroup for its softmax, one
// thread a row, while the tensor cores are busy with the other's products:
//   warps 0-3, 4-7  softmax of A and B (a thread holds a row's 128 scores)
//   warp 8          the products, issued by the warp in step, one elected lane
//   warp 9          the copies (TMA: one box per page and 64 dims; FP8: bulk
//                   copies of codes and scales)
//   warps 10, 11    make the V tiles safe (below); FP8: warps 10-15, which
//                   also turn E4M3 pages into bf16 tiles
// The running maximum is only raised (and O rescaled, which takes a TMEM round
// trip) when a row's maximum has grown by more than 2^8: the weights are then
// at most 2^8, which costs no precision in bf16 and 32 bits.
//
// Rounding.  Q and K products are exact, sums 32-bit; P is rounded once to
// bf16 (2^-8 of each weight; its errors average out over the tokens, and the
// output is rounded to the same 8 bits).  The sum of weights is taken from
// the unrounded ones.  FP8: codes become bf16 exactly, the key scales
// multiply S, the value scales multiply P, in 32 bits.
//
// Masked values.  0 * NaN is NaN, so a V row that some rows of the tile must
// not see may not enter the product with NaN or infinities in it: rows of no
// token (past the length, holes) are zeroed, and where the mask cuts a tile the
// elements that are not finite are zeroed and the rows that do see them get
// them added at the end.  Tiles that all rows see whole need nothing of it.
//
// Work.  A piece (two row tiles of a kv head) goes to one CTA; the pieces, longest
// first, are dealt to one CTA per SM in rounds, to and fro.  Where the last round
// (or the only one) has a piece for every second CTA at most, its pieces are
// split along their tokens and a second kernel joins the parts, in order: 512
// pieces of 64 tiles on 152 SMs are three rounds and a half then, not four (420
// -> 384 us).  What the lengths are is read on the device.
//
// Measured (back to back in a graph): 8192 tokens, 16 / 4 heads of 128, all of a
// prefix of 7411 seen: 374 us, 1.34 PFLOP/s; 8192 causal tokens 218, and of 64 / 8
// heads of 64 699 us, 0.79 PFLOP/s (a token and row cost the same exponential and
// half the products), over FP8 pages 384 and 1019; three chunks over FP8 pages 735,
// 0.52 PFLOP/s; four ragged chunks of 120 tokens 21.9 us.  What bounds it: with 128
// dims the chain S, softmax, P V, next S of a row tile, of which the other tile's
// covers a part (products alone, with the same handshakes, take 172 us where the
// kernel takes 218); with 64 dims the softmax warps' own time (two thirds of a
// tile's 3000 cycles), which is latency: two warps a scheduler, each with a serial
// run over 128 scores, leave the issue slots half empty (47% busy; tensor pipe and
// special functions 34%).  FP8: the softmax threads read 256 scales a tile and row
// from shared memory, six warps convert 2 x 128 rows a tile, and both share the
// issue slots (59% busy).  Exponentials left out (to see) change 0 with 128 dims
// and 7% with 64.  Registers spilled a thread: 156 bytes (bf16, 128 dims; with a
// cap or bias up to 224), 312 to 372 (FP8, 128 dims), 136 to 196 (FP8, 64), 0 to 36
// (bf16, 64).
#include <cmath>
#include <type_traits>

#include "launch.h"
#include "paged.cuh"
#include "tensor_map.h"

namespace tt {
namespace {

constexpr int kRows = 128;   // rows of a row tile
constexpr int kKeys = 128;   // tokens of a K / V tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kFixWarp = 10;
constexpr int kCounters = 1024;  // the decode kernel's, at the workspace's start: left alone
constexpr int kJoinBytes = (kCounters + 1) * 16;
constexpr int kMaxSplit = 32;
constexpr int kMaxSorted = 64;   // sequences that are put in order of length
constexpr int kTailTiles = 8;    // tiles a piece of the last round has to have to be split
constexpr uint32_t kAll = 0xffffffffu;

template <int D, bool FP8>
struct Plan {
  // warps 0-7 softmax, 8 products, 9 copies, and from kFixWarp on those that
  // make the V tiles safe: two; FP8: six, which convert.  Registers a thread:
  // at launch, for the softmax warps (a thread holds a row's 128 scores), for
  // the others (bf16 208 / 88: 383 us for the 370 below, 232 / 40: 381; FP8 200 /
  // 56: 744 for 731, 216 / 40: 754).
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kFixers = kThreads - 32 * kFixWarp;
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
  static constexpr int kOffKv = 2 * kTile;
  static constexpr int kOffRaw = kOffKv + kSlots * kTile;
  static constexpr int kOffScale = kOffRaw + kRaws * kRaw;      // [4 tiles][key, value][128]
  static constexpr int kOffLine = kOffScale + (FP8 ? 4 * 2 * kKeys * 4 : 0);
  static constexpr int kOffStart = kOffLine + (kPagedMaxBatch + 4) * 4;
  static constexpr int kOffEnd = kOffStart + kPagedMaxBatch * 4;
  static constexpr int kOffLen = kOffEnd + kPagedMaxBatch * 4;
  static constexpr int kOffOrder = kOffLen + kPagedMaxBatch * 4;
  static constexpr int kOffBar = kOffOrder + kPagedMaxBatch * 4;
  static constexpr int kSmem = 1024 + kOffBar + 640;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOffBar % 8 == 0, "barriers");
  // TMEM columns of A and B: S, O and P.  With 128 dims P lies over S (all
  // 512 columns are taken) and the next scores wait for P V; with 64 it has
  // its own, and they wait only until S is read.
  static constexpr bool kOwnP = D == 64;
  __host__ __device__ static constexpr int kColS(int g) { return 128 * g; }
  __host__ __device__ static constexpr int kColO(int g) { return 256 + D * g; }
  __host__ __device__ static constexpr int kColP(int g) { return kOwnP ? 384 + 64 * g : kColS(g); }
};

struct PrefillArgs {
  const int32_t* starts;
  int64_t tokens;
  int group, per_tile;  // heads per kv head, tokens per row tile
  float scale, softcap;
  int window;
  const float* slopes;
  const float* sinks;
  const int32_t* prefix;
  uint16_t* out;
  float* lse;
  bool may_split;   // the join kernel follows
  int4* joins;      // for it: [0].x the pieces, then a record per piece and row tile
  float* parts;
  int32_t* err;
};

// ---- tcgen05
__device__ __forceinline__ uint64_t desc_base() {
  return (uint64_t(1024 >> 4) << 32)  // stride: 8 rows of 128 bytes
         | (uint64_t(1) << 46)        // descriptor version
         | (uint64_t(2) << 61);       // 128-byte swizzle
}
// K-major operand (rows of 64 contiguous elements of the contraction).
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return desc_base() | (uint64_t(1) << 16) | uint64_t((addr >> 4) & 0x3fffu);
}
// MN-major operand (rows = steps of the contraction); `leading` bytes from
// one 64-element span of the outer dimension to the next.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t leading) {
  return desc_base() | (uint64_t(leading >> 4) << 16) | uint64_t((addr >> 4) & 0x3fffu);
}
// bf16 x bf16 -> f32, 128 rows, n columns; mn: B is MN-major.
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
         (uint32_t(kRows >> 4) << 24);
}
// The products are issued by a whole warp in step, one elected lane each:
// the compiler then knows that their operands are the same in all lanes and
// keeps them in uniform registers.  (In a branch of one lane every operand is
// moved there first: 60 to 110 cycles an instruction, more than the products
// themselves take.)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar)
      : "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// Waits for this thread's tcgen05.ld; the registers pass through, so that
// nothing that uses them is moved before it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                 "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this warp's 32 lanes (complete after wait_ld).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// 64 columns of this warp's 32 lanes into r[first ..] (complete after
// wait_ld128).
template <int first>
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17,"
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33,"
      "%34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49,"
      "%50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(r[first + 0]), "=r"(r[first + 1]), "=r"(r[first + 2]), "=r"(r[first + 3]), "=r"(r[first + 4]), "=r"(r[first + 5]), "=r"(r[first + 6]),
      "=r"(r[first + 7]), "=r"(r[first + 8]), "=r"(r[first + 9]), "=r"(r[first + 10]), "=r"(r[first + 11]), "=r"(r[first + 12]), "=r"(r[first + 13]),
      "=r"(r[first + 14]), "=r"(r[first + 15]), "=r"(r[first + 16]), "=r"(r[first + 17]), "=r"(r[first + 18]), "=r"(r[first + 19]), "=r"(r[first + 20]),
      "=r"(r[first + 21]), "=r"(r[first + 22]), "=r"(r[first + 23]), "=r"(r[first + 24]), "=r"(r[first + 25]), "=r"(r[first + 26]), "=r"(r[first + 27]),
      "=r"(r[first + 28]), "=r"(r[first + 29]), "=r"(r[first + 30]), "=r"(r[first + 31]), "=r"(r[first + 32]), "=r"(r[first + 33]), "=r"(r[first + 34]),
      "=r"(r[first + 35]), "=r"(r[first + 36]), "=r"(r[first + 37]), "=r"(r[first + 38]), "=r"(r[first + 39]), "=r"(r[first + 40]), "=r"(r[first + 41]),
      "=r"(r[first + 42]), "=r"(r[first + 43]), "=r"(r[first + 44]), "=r"(r[first + 45]), "=r"(r[first + 46]), "=r"(r[first + 47]), "=r"(r[first + 48]),
      "=r"(r[first + 49]), "=r"(r[first + 50]), "=r"(r[first + 51]), "=r"(r[first + 52]), "=r"(r[first + 53]), "=r"(r[first + 54]), "=r"(r[first + 55]),
      "=r"(r[first + 56]), "=r"(r[first + 57]), "=r"(r[first + 58]), "=r"(r[first + 59]), "=r"(r[first + 60]), "=r"(r[first + 61]), "=r"(r[first + 62]),
      "=r"(r[first + 63])
      : "r"(addr));
}
// Waits for this thread's loads; the registers pass through, so that nothing
// that uses them is moved before.
__device__ __forceinline__ void wait_ld128(uint32_t (&r)[128]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
      "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
      "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
      "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
      "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]),
      "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]),
      "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]),
      "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
      "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]),
      "+r"(r[63])
      :
      : "memory");
  asm volatile(""
      : "+r"(r[64]), "+r"(r[65]), "+r"(r[66]), "+r"(r[67]), "+r"(r[68]), "+r"(r[69]), "+r"(r[70]),
      "+r"(r[71]), "+r"(r[72]), "+r"(r[73]), "+r"(r[74]), "+r"(r[75]), "+r"(r[76]), "+r"(r[77]),
      "+r"(r[78]), "+r"(r[79]), "+r"(r[80]), "+r"(r[81]), "+r"(r[82]), "+r"(r[83]), "+r"(r[84]),
      "+r"(r[85]), "+r"(r[86]), "+r"(r[87]), "+r"(r[88]), "+r"(r[89]), "+r"(r[90]), "+r"(r[91]),
      "+r"(r[92]), "+r"(r[93]), "+r"(r[94]), "+r"(r[95]), "+r"(r[96]), "+r"(r[97]), "+r"(r[98]),
      "+r"(r[99]), "+r"(r[100]), "+r"(r[101]), "+r"(r[102]), "+r"(r[103]), "+r"(r[104]),
      "+r"(r[105]), "+r"(r[106]), "+r"(r[107]), "+r"(r[108]), "+r"(r[109]), "+r"(r[110]),
      "+r"(r[111]), "+r"(r[112]), "+r"(r[113]), "+r"(r[114]), "+r"(r[115]), "+r"(r[116]),
      "+r"(r[117]), "+r"(r[118]), "+r"(r[119]), "+r"(r[120]), "+r"(r[121]), "+r"(r[122]),
      "+r"(r[123]), "+r"(r[124]), "+r"(r[125]), "+r"(r[126]), "+r"(r[127])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st64(uint32_t addr, const uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x64.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18,"
      "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34,"
      "%35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50,"
      "%51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, %64};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(r[32]), "r"(r[33]), "r"(r[34]), "r"(r[35]),
      "r"(r[36]), "r"(r[37]), "r"(r[38]), "r"(r[39]), "r"(r[40]), "r"(r[41]), "r"(r[42]),
      "r"(r[43]), "r"(r[44]), "r"(r[45]), "r"(r[46]), "r"(r[47]), "r"(r[48]), "r"(r[49]),
      "r"(r[50]), "r"(r[51]), "r"(r[52]), "r"(r[53]), "r"(r[54]), "r"(r[55]), "r"(r[56]),
      "r"(r[57]), "r"(r[58]), "r"(r[59]), "r"(r[60]), "r"(r[61]), "r"(r[62]), "r"(r[63])
      : "memory");
}

__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, int x, int h, int t,
                                      uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Two 32-bit lanes at once.
__device__ __forceinline__ uint64_t f2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  return f2(__float_as_uint(lo), __float_as_uint(hi));
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two E4M3 codes (low 16 bits) -> bf16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(h)
      : "r"(w));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return bf16x2(f.x, f.y);
}

// What one piece of work is: the row tiles A and B of q tile `qt` of sequence
// b, kv head j, the part [k0, k1) of its K / V tiles.
struct Item {
  int b, j, len, pre;
  int tok0, new_tokens;  // first flat token of tile A; the sequence's tokens from it on
  int p0;                // place of tok0
  int lo, hi;            // tokens that some row sees
  int all_lo, all_hi;    // tokens that every row sees
  int k0, k1, parts, part;
  int base;              // number among the joined pieces, or -1
};

// Waits for a phase; gives up after kWaitLimitNs, or when another thread has.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* quit,
                                     int32_t* err) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(a, parity)) return true;
    if ((it & 15u) == 0u) {
      if (*quit) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *quit = 1;
        flag_error(err, kErrTimeout);
        return false;
      }
    }
  }
}

// Which of the 32 dims from d0 on have a value of +infinity, -infinity, NaN (a
// bit each) among the tokens [lo, hi) of sequence b and kv head j, in the tiles
// whose values were kept out of the product: those that the mask cuts (not
// within [all_lo, all_hi)), and with `holes` those of which pages are missing.
// Only these are read, a page looked up once: one NaN in a cut tile of 2500
// tokens behind 17,000 (16 / 4 heads of 128) costs 0.17 ms.  (The whole row,
// element by element, took 45 ms, and would have been past a wait's limit for
// some 400,000 tokens.  Every element taken apart, not only those of rows that
// have one that is not finite: 0.40 ms.)
template <int D, bool FP8>
__device__ __noinline__ uint3 not_finite(const PagedKv& kv, int b, int j, int lo, int hi,
                                         int all_lo, int all_hi, bool holes, int d0) {
  uint3 x = make_uint3(0u, 0u, 0u);
  const int rows = 1 << kv.page_shift;
  for (int t0 = lo / kKeys * kKeys; t0 < hi; t0 += kKeys) {
    if (t0 >= all_lo && t0 + kKeys <= all_hi) {
      bool whole = true;
      for (int t = t0; holes && t < t0 + kKeys; t += rows) whole &= paged_page(kv, b, t, nullptr) >= 0;
      if (whole) continue;
    }
    for (int tp = t0; tp < t0 + kKeys; tp += rows) {
      const int from = max(tp, lo), n = min(tp + rows, hi) - from;
      if (n <= 0) continue;
      const int page = paged_page(kv, b, tp, nullptr);
      if (page < 0) continue;
      const int64_t at = paged_row(kv, page, j, from);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.v) +
                                                        (at * D + d0) * (FP8 ? 1 : 2));
#pragma unroll 4
      for (int t = 0; t < n; ++t) {
        // carries into the top bits of bytes 0x7f and 0xff (NaN), or of halves whose
        // exponent is all ones: almost always none, and the row is done with
        uint4 q[FP8 ? 2 : 4];
        uint32_t any = 0u;
#pragma unroll
        for (int u = 0; u < (FP8 ? 2 : 4); ++u) {
          q[u] = __ldcg(src + t * (D / (FP8 ? 16 : 8)) + u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t c = reinterpret_cast<const uint32_t*>(&q[u])[i];
            any |= FP8 ? (c & 0x7f7f7f7fu) + 0x01010101u : (c & 0x7f807f80u) + 0x00800080u;
          }
        }
        if constexpr (FP8) {  // a scale that is not finite makes all of the row so
          if (!(fabsf(__ldcg(kv.v_scales + at + t)) <= kFiniteMax)) x.z = kAll;
        }
        if (!(any & (FP8 ? 0x80808080u : 0x80008000u))) continue;
#pragma unroll
        for (int d = 0; d < 32; ++d) {
          if constexpr (FP8) {
            const uint32_t v = reinterpret_cast<const uint32_t*>(q)[d / 4] >> (8 * (d & 3));
            x.z |= uint32_t((v & 0x7fu) == 0x7fu) << d;
          } else {
            const uint32_t v = reinterpret_cast<const uint32_t*>(q)[d / 2] >> (16 * (d & 1)) & 0xffffu;
            x.x |= uint32_t(v == 0x7f80u) << d;
            x.y |= uint32_t(v == 0xff80u) << d;
            x.z |= uint32_t((v & 0x7fffu) > 0x7f80u) << d;
          }
        }
      }
    }
  }
  return x;
}

// What is done to the scores: nothing but a positive scale; a cap, a bias or
// another scale (the plain kernel's loop stays short without them); a large cap.
enum Scores { kPlain, kGeneral, kLargeCap };
template <int D, bool FP8, Scores SC>
__global__ void __launch_bounds__(Plan<D, FP8>::kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ PagedKv kv,
                         const PrefillArgs a) {
  using P = Plan<D, FP8>;
  constexpr bool GEN = SC != kPlain;
  constexpr int kThreads = P::kThreads, kFixers = P::kFixers;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + P::kOffScale);
  // of the i-th sequence taken: the q tiles before it, its first flat token and
  // the one after its last, its length, its number
  int32_t* line = reinterpret_cast<int32_t*>(smem + P::kOffLine);
  int32_t* first = reinterpret_cast<int32_t*>(smem + P::kOffStart);
  int32_t* ends = reinterpret_cast<int32_t*>(smem + P::kOffEnd);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + P::kOffLen);
  int32_t* order = reinterpret_cast<int32_t*>(smem + P::kOffOrder);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kOffBar);
  uint64_t* empty = full + P::kSlots;
  uint64_t* ready = empty + P::kSlots;   // slot made safe, or converted
  uint64_t* raw_full = ready + P::kSlots;
  uint64_t* raw_empty = raw_full + 4;
  uint64_t* q_full = raw_empty + 4;      // [2]
  uint64_t* q_free = q_full + 2;
  uint64_t* s_full = q_free + 1;         // [2]
  uint64_t* p_full = s_full + 2;         // [2]
  uint64_t* o_done = p_full + 2;         // [2]
  uint64_t* s_read = o_done + 2;         // [2]
  uint64_t* drained = s_read + 2;
  uint32_t* have = reinterpret_cast<uint32_t*>(drained + 1);  // [8] boxes present, per tile
  int* dirty = reinterpret_cast<int*>(have + 8);              // [4] item number + 1
  int* misc = dirty + 4;  // [0] TMEM address, [1] quit, [4 .. 19] scan
  volatile int* quit = misc + 1;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P::kSlots; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 2);  // both row tiles
      mbar_init(smem_u32(&ready[i]), kFixers);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), kFixers);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&q_full[g]), 1);
      mbar_init(smem_u32(&s_full[g]), 1);
      mbar_init(smem_u32(&p_full[g]), kRows);
      mbar_init(smem_u32(&o_done[g]), 1);
      mbar_init(smem_u32(&s_read[g]), kRows);
    }
    mbar_init(smem_u32(q_free), 2);
    mbar_init(smem_u32(drained), 1);
    for (int i = 0; i < 4; ++i) dirty[i] = 0;
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

  // ---- the pieces of work: q tiles of every sequence, scanned.  Where there are
  // more than about one for every CTA, the sequences are taken in order of their
  // lengths, so that the longest pieces come first (three ragged chunks of 64
  // heads of 64 over FP8 pages: 746 us, in the order given 790); up to 64 of
  // them, as each is ranked against all.
  const int64_t tokens = a.tokens;
  auto start_of = [&](int b) {
    const int64_t s = __ldcg(a.starts + b);
    return int(s < 0 ? 0 : s > tokens ? tokens : s);
  };
  for (int b = tid; b < kv.batch; b += kThreads) {
    first[b] = start_of(b);
    ends[b] = start_of(b + 1);
    order[b] = b;
    lens[b] = paged_len(kv, b, blockIdx.x == 0 ? a.err : nullptr);
  }
  __syncthreads();
  const bool sorted = kv.batch > 1 && kv.batch <= kMaxSorted &&
                      tokens * kv.kv_heads > int64_t(2) * a.per_tile * gridDim.x;
  if (sorted) {
    int rank = 0, s0 = 0, s1 = 0, n = 0;
    if (tid < kv.batch) {
      s0 = first[tid], s1 = ends[tid], n = lens[tid];
      for (int c = 0; c < kv.batch; ++c) rank += lens[c] < n || (lens[c] == n && c < tid);
    }
    __syncthreads();
    if (tid < kv.batch) first[rank] = s0, ends[rank] = s1, lens[rank] = n, order[rank] = tid;
    __syncthreads();
  }
  {
    constexpr int kPer = (kPagedMaxBatch + kThreads - 1) / kThreads;
    const int per = (kv.batch + kThreads - 1) / kThreads;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mine[i] = 0;
      if (i < per && tid * per + i < kv.batch) {
        const int n = ends[tid * per + i] - first[tid * per + i];
        mine[i] = n > 0 ? (n + 2 * a.per_tile - 1) / (2 * a.per_tile) : 0;
      }
      sum += mine[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) misc[4 + warp] = run;
    __syncthreads();
    int before = run - sum;
    for (int w = 0; w < warp; ++w) before += misc[4 + w];
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
  const int tiles = line[kv.batch];
  const int pieces = tiles * kv.kv_heads;  // (tokens x heads fit 31 bits)
  const int sms = gridDim.x;
  const int G = a.group, heads = G * kv.kv_heads, TT = a.per_tile;
  // Whole rounds of pieces, then the rest: where it has a piece for every second
  // CTA at most, its pieces are split along their tokens.
  const int whole = pieces / sms * sms;
  const int rest = pieces - whole;
  int split = a.may_split && rest > 0 && rest * 2 <= sms ? sms / rest : 1;
  split = split < kMaxSplit ? split : kMaxSplit;

  auto item_of = [&](int idx) {
    Item w;
    int piece = idx;
    w.part = 0;
    w.base = -1;
    if (split > 1 && idx >= whole) {
      w.base = (idx - whole) / split;
      w.part = idx - whole - w.base * split;
      piece = whole + w.base;
    }
    w.j = piece % kv.kv_heads;
    const int u = tiles - 1 - piece / kv.kv_heads;  // the longest first
    int lo = 0, hi = kv.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (line[mid] <= u) lo = mid; else hi = mid;
    }
    w.b = order[lo];
    const int s0 = first[lo], s1 = ends[lo];
    const int q0 = (u - line[lo]) * 2 * TT;
    w.tok0 = s0 + q0;
    w.new_tokens = s1 - w.tok0;
    w.len = lens[lo];
    w.p0 = w.len - w.new_tokens;
    w.pre = a.prefix ? __ldcg(a.prefix + w.b) : 0;
    const int rows = w.new_tokens < 2 * TT ? w.new_tokens : 2 * TT;
    const int plast = w.p0 + rows - 1;
    int top = plast + 1 > w.pre ? plast + 1 : w.pre;
    top = top < w.len ? top : w.len;
    w.hi = plast < 0 ? 0 : top;
    const int pf = w.p0 > 0 ? w.p0 : 0;  // the first row with a place
    w.lo = a.window > 0 && pf + 1 > a.window ? pf + 1 - a.window : 0;
    if (w.lo > w.hi) w.lo = w.hi;
    w.all_hi = w.p0 < 0 ? 0 : w.p0 + 1 > w.pre ? w.p0 + 1 : w.pre;
    w.all_hi = w.all_hi < w.hi ? w.all_hi : w.hi;
    w.all_lo = a.window > 0 && plast + 1 > a.window ? plast + 1 - a.window : 0;
    const int ka = w.lo / kKeys, kb = (w.hi + kKeys - 1) / kKeys;
    const int nk = w.hi > w.lo ? kb - ka : 0;
    // two tiles a part at least (a part's start costs about as much)
    const int most = nk > 3 ? nk / 2 : 1;
    w.parts = w.base < 0 ? 1 : split < most ? split : most;
    w.k0 = w.k1 = ka;
    if (w.part < w.parts) {
      w.k0 = ka + int(int64_t(nk) * w.part / w.parts);
      w.k1 = ka + int(int64_t(nk) * (w.part + 1) / w.parts);
    }
    return w;
  };
  auto has_b = [&](const Item& w) { return w.new_tokens > TT; };
  // After whole rounds a split gains less than a round, and costs the parts' way
  // through memory: short pieces stay whole.
  if (split > 1 && whole > 0) {
    const Item w = item_of(whole);
    const int nk = (w.hi + kKeys - 1) / kKeys - w.lo / kKeys;
    if (nk < kTailTiles) split = 1;
  }
  const int items = whole + rest * split;
  if (a.may_split && blockIdx.x == 0 && tid == 0)
    a.joins[0] = make_int4(split > 1 ? rest : 0, split, 0, 0);
  // The CTA's turns: the items, longest first, are dealt to the CTAs to and
  // fro, which evens out what a falling order leaves uneven; -1 at the end.
  auto turn_of = [&](int turn) {
    if (turn * sms >= items) return -1;
    return turn * sms + (turn & 1 ? sms - 1 - int(blockIdx.x) : int(blockIdx.x));
  };
  const int br_shift = kv.page_shift;  // rows of a box: a page, 16 .. 128
  const int boxes = kKeys >> br_shift;

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::kOtherRegs));
    if (warp == kLoadWarp) {
      // ============================================================ copies
      uint32_t n = 0;  // slots used
      int seq = 0;     // items done
      uint32_t nt = 0; // tiles
      bool ok = true;
      for (int turn = 0, idx; ok && (idx = turn_of(turn)) >= 0; ++turn) {
        if (idx >= items) continue;
        const Item w = item_of(idx);
        if (w.k1 <= w.k0) continue;
        const int groups = has_b(w) ? 2 : 1;
        // Q is free when the last score products of the item before are done
        if (seq > 0) ok = __all_sync(kAll, wait(q_free, uint32_t(seq - 1) & 1u, quit, a.err));
        if (!ok) break;
        if (lane < groups) {
          const uint32_t bar = smem_u32(&q_full[lane]);
          mbar_arrive_expect_tx(bar, uint32_t(TT * G * 128 * P::kHalves));
          for (int h = 0; h < P::kHalves; ++h)
            tma_q(sbase + lane * P::kTile + h * P::kSpan, &map_q, 64 * h, w.j * G,
                  w.tok0 + lane * TT, bar);
        }
        __syncwarp();
        ++seq;
        auto look = [&](int kt) {
          const int t = kt * kKeys + (lane << br_shift);
          const bool in = lane < boxes && t < w.hi && t + (1 << br_shift) > w.lo;
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
        for (int g = 0; g < 2; ++g) (void)mbar_wait_bounded(smem_u32(&q_full[g]), uint32_t(seq - 1) & 1u);
      }
    } else if (warp == kMmaWarp) {
      // ========================================================== products
      // One warp for both row tiles, whichever is ready, so that a tile's
      // products (P V, then the next scores) go to the tensor cores in one
      // piece.  (With an issuer for each they are taken in turn, both tiles
      // wait for both, and softmax and products do not overlap: a softmax
      // warp waited 2275 of 4190 cycles a tile.)  One commit a tile: products
      // finish in order, so scores that are there say that the P V before
      // them is done.
      const uint32_t kv0 = sbase + P::kOffKv;
      uint32_t n = 0, my0 = 0, my1 = 0, seq0 = 0, seq1 = 0;  // slots; tiles, items of A and B
      bool ok = tmem == 0;  // all columns are ours, so they begin at 0
      if (!ok && lane == 0) {
        *quit = 1;
        flag_error(a.err, kErrShape);
      }
      auto scores = [&](auto gc, uint32_t slot) {
        constexpr int g = decltype(gc)::value;
        const uint64_t q = desc_k(sbase + g * P::kTile), k = desc_k(kv0 + slot * P::kTile);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t off = ((i >> 2) * P::kSpan + (i & 3) * 32) >> 4;
          mma_ss(P::kColS(g), q + off, k + off, idesc(kKeys, false), i > 0);
        }
        commit(smem_u32(&s_full[g]));
      };
      auto values = [&](auto gc, uint32_t slot, uint32_t more) {
        constexpr int g = decltype(gc)::value;
        const uint64_t v = desc_mn(kv0 + slot * P::kTile, P::kHalves > 1 ? P::kSpan : 1024);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(P::kColO(g), P::kColP(g) + 8 * k, v + k * (2048 >> 4),
                 idesc(D, true), k > 0 ? 1u : more);
      };
      // slot use m has its K tile, its V tile (bf16: an even number of slots,
      // so that a slot is K's or V's for good)
      auto key_bar = [&](uint32_t m) {
        return smem_u32(FP8 ? &ready[m % P::kSlots] : &full[m % P::kSlots]);
      };
      auto phase = [&](uint32_t m) { return (m / P::kSlots) & 1u; };
      using G0 = std::integral_constant<int, 0>;
      using G1 = std::integral_constant<int, 1>;
      for (int turn = 0, idx; ok && (idx = turn_of(turn)) >= 0; ++turn) {
        if (idx >= items) continue;
        const Item w = item_of(idx);
        const int nk = __shfl_sync(kAll, w.k1 - w.k0, 0);
        if (nk <= 0) continue;
        const bool b = __shfl_sync(kAll, int(has_b(w)), 0) != 0;
        ok = __all_sync(kAll, wait(&q_full[0], seq0++ & 1u, quit, a.err) &&
                                  wait(FP8 ? &ready[n % P::kSlots] : &full[n % P::kSlots],
                                       phase(n), quit, a.err));
        if (!ok) break;
        fence_after();
        scores(G0{}, n % P::kSlots);
        if (b) {
          ok = __all_sync(kAll, wait(&q_full[1], seq1++ & 1u, quit, a.err));
          if (!ok) break;
          fence_after();
          scores(G1{}, n % P::kSlots);
        }
        // of each row tile: products P V issued, scores issued
        uint32_t v0 = 0, v1 = b ? 0 : nk, s0 = 1, s1 = b ? 1 : nk;
        uint64_t since = 0;  // of the idle stretch
        auto tile = [&](auto gc, uint32_t& vi, uint32_t& si, uint32_t& my) {
          constexpr int g = decltype(gc)::value;
          bool did = false;
          const uint32_t m = n + 2 * vi;
          if (vi < uint32_t(nk)) {
            const bool next = vi + 1 < uint32_t(nk);
            const bool go =
                mbar_test_wait(smem_u32(&p_full[g]), my & 1u) &&
                mbar_test_wait(smem_u32(&ready[(m + 1) % P::kSlots]), phase(m + 1)) &&
                (P::kOwnP || !next || mbar_test_wait(key_bar(m + 2), phase(m + 2)));
            if (__all_sync(kAll, go)) {
              fence_after();
              values(gc, (m + 1) % P::kSlots, vi > 0);
              if (P::kOwnP || !next) commit(smem_u32(&o_done[g]));
              if (!P::kOwnP && next) scores(gc, (m + 2) % P::kSlots);
              ++vi;
              ++my;
              did = true;
            }
          }
          if constexpr (P::kOwnP) {
            // tile si's scores, once those before are read (my - vi tiles
            // were before this item)
            if (si < uint32_t(nk)) {
              const uint32_t ms = n + 2 * si;
              const bool go = mbar_test_wait(smem_u32(&s_read[g]), (my - vi + si - 1) & 1u) &&
                              mbar_test_wait(key_bar(ms), phase(ms));
              if (__all_sync(kAll, go)) {
                fence_after();
                scores(gc, ms % P::kSlots);
                ++si;
                did = true;
              }
            }
          }
          return did;
        };
        for (uint32_t idle = 0; v0 < uint32_t(nk) || v1 < uint32_t(nk);) {
          bool did = tile(G0{}, v0, s0, my0);
          did |= tile(G1{}, v1, s1, my1);
          if (did) {
            idle = 0;
          } else if ((++idle & 63u) == 0u) {  // (a sleep of 20 ns here: 222 us for 218.5)
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
      for (int turn = 0, idx; ok && (idx = turn_of(turn)) >= 0; ++turn) {
        if (idx >= items) continue;
        const Item w = item_of(idx);
        if (w.k1 <= w.k0) continue;
        ++seq;
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++nt) {
          const int t0 = kt * kKeys;
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
              const bool cut = t0 < w.all_lo || t0 + kKeys > w.all_hi;
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
                    if (t < w.lo || t >= w.hi || !((got >> (r >> br_shift)) & 1u)) {
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
                    if (t < w.lo || t >= w.hi || !((got >> (r >> br_shift)) & 1u)) {
                      v = 0.f;
                    } else if (i >= kKeys && !(fabsf(v) <= 3.4028234663852886e38f)) {
                      v = 0.f;  // a value row that some must not see: as an element of V
                      bad = true;
                    }
                  }
                  scales[(nt & 3u) * 2 * kKeys + i] = v;
                }
              }
              if (bad) dirty[seq & 3] = seq;
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              mbar_arrive(smem_u32(&raw_empty[rs]));
              mbar_arrive(smem_u32(&ready[s]));
            } else {
              if (part == 0) continue;  // K: scores of masked tokens are replaced
              ok = wait(&full[s], turn & 1u, quit, a.err);
              if (!ok) break;
              const uint32_t got = have[nt & 7u];
              const bool cut = t0 < w.all_lo || t0 + kKeys > w.all_hi;
              if (cut || got != kAll >> (32 - boxes)) {
                bool bad = false;
                for (int r = ft; r < kKeys; r += kFixers) {
                  const int t = t0 + r;
                  const bool none =
                      t < w.lo || t >= w.hi || !((got >> (r >> br_shift)) & 1u);
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
                if (bad) dirty[seq & 3] = seq;
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
    uint32_t nt = 0, my = 0;  // tiles of the CTA; tiles of this row tile
    uint32_t slot = 0, done = 0;  // slot uses of the CTA; items of this row tile
    int seq = 0;
    bool ok = true;
    for (int turn = 0, idx; ok && (idx = turn_of(turn)) >= 0; ++turn) {
      if (idx >= items) continue;
      const Item w = item_of(idx);
      if (w.part >= w.parts) continue;
      const int nk = w.k1 - w.k0;
      if (nk > 0) ++seq;
      const int tok = g * TT + rt;  // among the item's tokens
      const bool mine = rt < TT && tok < w.new_tokens;
      const int groups = has_b(w) ? 2 : 1;
      if (w.base >= 0 && w.part == 0 && r == 0 && (w.parts == 1 || (g == 1 && groups == 1)))
        a.joins[1 + 2 * w.base + g] = make_int4(0, 0, 0, 0);
      if (g == 1 && groups == 1) {
        nt += nk;
        slot += 2 * nk;
        continue;
      }
      const int p = w.p0 + tok, h = w.j * G + rh;
      // the tokens this row sees; a row of no token takes whatever comes
      int rhi = 0x7fffffff, rlo = 0;
      if (mine) {
        rhi = p < 0 ? 0 : p + 1 > w.pre ? p + 1 : w.pre;
        rhi = rhi < w.len ? rhi : w.len;
        rlo = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
      }
      const float slope = a.slopes && mine ? __ldcg(a.slopes + h) * kLog2e : 0.f;
      // one arrival of each row tile; the only row tile of an item arrives for both
      auto free_slot = [&](uint32_t use) {
        if (r == 0)
          for (int e = groups; e <= 2; ++e) mbar_arrive(smem_u32(&empty[use % P::kSlots]));
      };
      float m = -INFINITY, l = 0.f;
      bool holes = false;  // pages missing of a tile that the mask does not cut
      for (int i = 0; i < nk; ++i, ++nt, ++my) {
        ok = __all_sync(kAll, wait(&s_full[g], my & 1u, quit, a.err));
        if (!ok) break;
        fence_after();
        // these scores are there: their K tile is done with, and where they
        // waited for it the V tile before
        free_slot(slot);
        if (!P::kOwnP && i > 0) free_slot(slot - 1);
        if (i + 1 == nk && r == 0)
          for (int e = groups; e <= 2; ++e) mbar_arrive(smem_u32(q_free));
        slot += 2;
        [[maybe_unused]] bool seen_o = false;
        const int t0 = (w.k0 + i) * kKeys;
        const uint32_t got = have[nt & 7u];
        const bool whole = got == kAll >> (32 - boxes);
        holes |= !whole && t0 >= w.all_lo && t0 + kKeys <= w.all_hi;
        const bool clear = __all_sync(kAll, t0 >= rlo && t0 + kKeys <= rhi) && whole;
        const float* ks = scales + ((nt & 3u) * 2) * kKeys;
        // All of the row's scores at once, and its weights at once: a TMEM access
        // takes hundreds of cycles whatever its size.  (Read twice in pieces of
        // 32 columns, for the maximum and for the weights: 1177 against 761 us at
        // 8192 tokens, 64 heads of 64; written in four pieces: 897.)
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
          {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + e);
              float f[4];
              un2(mul2(f2(x[e], x[e + 1]), f2(k.x, k.y)), f[0], f[1]);
              un2(mul2(f2(x[e + 2], x[e + 3]), f2(k.z, k.w)), f[2], f[3]);
#pragma unroll
              for (int u = 0; u < 4; ++u) x[e + u] = __float_as_uint(f[u]);
            }
          }
        };
        // a large cap, two scores at a time where all are below the series' end
        auto capped = [&](uint32_t* x) {
          float far = 0.f;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float v = __uint_as_float(x[e]) * mul;
            far = fmaxf(far, fabsf(v));
            x[e] = __float_as_uint(v);
          }
          if (__any_sync(kAll, far * cap.per >= kCapSeries)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              x[e] = __float_as_uint(cap_large(__uint_as_float(x[e]), cap));
            return;
          }
          auto both = [](float v) { return f2(v, v); };
          const uint64_t k = both(cap.per * kHalfLn2);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t s2 = f2(x[e], x[e + 1]), xc = mul2(s2, k), x2 = mul2(xc, xc);
            uint64_t p = fma2(x2, both(kCap4), both(kCap3));
            p = fma2(x2, p, both(kCap2));
            p = fma2(x2, p, both(kCap1));
            float v[2];
            un2(fma2(mul2(s2, x2), p, s2), v[0], v[1]);
            x[e] = __float_as_uint(v[0]);
            x[e + 1] = __float_as_uint(v[1]);
          }
        };
        // to log2 units, the long way: the cap, the bias, a scale <= 0
        auto general = [&](uint32_t* x, int c) {
          const float base = slope * float(t0 + 32 * c - p);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(x[e]);
            if constexpr (SC != kLargeCap) {
              v *= unit;
              if (a.softcap > 0.f) v = cap_small(v, cap);
            }
            x[e] = __float_as_uint(v + fmaf(slope, float(e), base));
          }
        };
        auto masked = [&](uint32_t* x, int c) {
          // this row's tokens of the columns, one bit each
          const int a0 = rlo - t0 - 32 * c, a1 = rhi - t0 - 32 * c;
          uint32_t see = a0 <= 0 ? kAll : a0 >= 32 ? 0u : kAll << a0;
          see &= a1 <= 0 ? 0u : a1 >= 32 ? kAll : kAll >> (32 - a1);
          if (!((got >> ((32 * c) >> br_shift)) & 1u)) see &= 0xffff0000u;
          if (!((got >> ((32 * c + 16) >> br_shift)) & 1u)) see &= 0x0000ffffu;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1u)) x[e] = 0xff800000u;
        };
        if constexpr (FP8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) scaled(s + 32 * c, c);
        }
        if constexpr (GEN) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if constexpr (SC == kLargeCap) capped(s + 32 * c);
            general(s + 32 * c, c);
          }
        }
        if (__builtin_expect(!clear, 0)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) masked(s + 32 * c, c);
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
        if constexpr (P::kOwnP) {  // the weights before these are read, their V tile done with
          if (!seen_o) {
            ok = __all_sync(kAll, i == 0 || wait(&o_done[g], (my - 1) & 1u, quit, a.err));
            if (!ok) break;
            fence_after();
          }
          if (i > 0) free_slot(slot - 3);
        }
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

      // ---- the item's end
      if (nk > 0) {
        ok = __all_sync(kAll, wait(&o_done[g], (P::kOwnP ? my - 1 : done++) & 1u, quit, a.err));
        if (!ok) break;
        fence_after();
        free_slot(slot - 1);
      }
      const int64_t row = int64_t(w.tok0 + tok) * heads + h;
      const bool poisoned = nk > 0 && *static_cast<volatile int*>(&dirty[seq & 3]) == seq;
      auto add_not_finite = [&](float* o, int d0) {
        const uint3 x = not_finite<D, FP8>(kv, w.b, w.j, max(rlo, w.k0 * kKeys),
                                           min(rhi, w.k1 * kKeys), w.all_lo, w.all_hi, holes, d0);
#pragma unroll
        for (int d = 0; d < 32; ++d) {
          if ((x.x >> d) & 1u) o[d] += INFINITY;
          if ((x.y >> d) & 1u) o[d] -= INFINITY;
          if ((x.z >> d) & 1u) o[d] = NAN;
        }
      };
      auto store = [&](const float* o, int c, float inv) {  // 32 dims from 32 c on
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + 32 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dst[e] = make_uint4(bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                              bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                              bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                              bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
      };
      if (w.parts == 1) {
        float inv = 0.f;
        if (mine) inv = close_row(m, l, a.sinks, h, a.lse, row);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (nk > 0) {
            tmem_ld32(to + 32 * c, o);
            wait_ld(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          float of[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) of[e] = __uint_as_float(o[e]);
          if (mine) {
            if (poisoned) add_not_finite(of, 32 * c);
            store(of, c, inv);
          }
        }
        fence_before();
        continue;
      }
      // a part: O [D / 4][128 rows] float4, max [128], sum [128]
      constexpr int kPartFloats = kRows * (D + 2);
      auto part_at = [&](int q) {
        return a.parts + (int64_t(w.base) * split + q) * 2 * kPartFloats + g * kPartFloats;
      };
      float* mypart = part_at(w.part);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(to + 32 * c, o);
        wait_ld(o);
        float of[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) of[e] = __uint_as_float(o[e]);
        if (mine && poisoned) add_not_finite(of, 32 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(mypart + ((8 * c + e) * kRows + r) * 4) =
              make_float4(of[4 * e], of[4 * e + 1], of[4 * e + 2], of[4 * e + 3]);
      }
      mypart[kRows * D + r] = m;
      mypart[kRows * (D + 1) + r] = l;
      if (w.part == 0 && r == 0) {
        const int left = w.new_tokens - g * TT;
        a.joins[1 + 2 * w.base + g] =
            make_int4(w.parts, w.tok0 + g * TT, left < TT ? left : TT, w.j);
      }
      fence_before();
    }
  }
  // ---- every role is done (or has given up): free the tensor memory
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// Joins the parts of split pieces, launched behind the kernel above: a block
// takes eight dims of a row tile at a time, a thread a row, with kJoin parts'
// loads in flight.  (Joined by the last CTA of a piece, 12 parts of a piece
// took 27 us: 1.6 MB through one SM.)
constexpr int kJoinThreads = kRows;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    paged_prefill_join_kernel(const PrefillArgs a, int heads) {
  constexpr int kJoin = 8;
  constexpr int kPartFloats = kRows * (D + 2);
  const int r = threadIdx.x;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int4 head = __ldcg(a.joins);
  const int units = head.x * 2 * (D / 8), split = head.y;
  const int rt = r / a.group, rh = r - rt * a.group;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = u / (D / 8), c = u % (D / 8);  // piece and row tile; dims 8c ..
    const int4 rec = __ldcg(a.joins + 1 + tile);    // parts, first token, tokens, kv head
    if (rt >= rec.z) continue;                      // (no parts: no tokens)
    const float* part = a.parts + (int64_t(tile >> 1) * split * 2 + (tile & 1)) * kPartFloats;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int q0 = 0; q0 < rec.x; q0 += kJoin) {
      float4 v[kJoin][2];
      float pm[kJoin], pl[kJoin], mx = m;
#pragma unroll
      for (int e = 0; e < kJoin; ++e) {
        const bool in = q0 + e < rec.x;
        const float* p = part + int64_t(in ? q0 + e : 0) * 2 * kPartFloats;
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

cudaError_t encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  if (enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dims,
          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

template <int D, bool FP8, Scores SC>
cudaError_t launch_as(const DeviceInfo& di, const PagedKv& kv, const PagedAttnArgs& a,
                      cudaStream_t s, bool pdl) {
  using P = Plan<D, FP8>;
  auto kern = paged_prefill_kernel<D, FP8, SC>;
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
  PrefillArgs d;
  d.starts = a.starts;
  d.tokens = a.tokens;
  d.group = G;
  d.per_tile = TT;
  d.scale = a.scale;
  d.softcap = a.softcap;
  d.window = a.window;
  d.slopes = a.slopes;
  d.sinks = a.sinks;
  d.prefix = a.prefix;
  d.out = a.out;
  d.lse = a.lse;
  // Whether a last round of half as many pieces as SMs or fewer is possible.
  // One sequence has this many pieces (tokens that it does not have only make this
  // too careful); several may have any number more, up to one q tile each.
  const int64_t pieces = (a.tokens + 2 * TT - 1) / (2 * TT) * kv.kv_heads;
  const int64_t rest = pieces % di.sms;
  d.may_split = kv.batch == 1 ? rest > 0 && rest * 2 <= di.sms
                              : pieces * 2 <= di.sms || pieces > di.sms;
  d.joins = reinterpret_cast<int4*>(static_cast<uint8_t*>(a.ws) + kCounters * 4);
  d.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kCounters * 4 + kJoinBytes);
  d.err = di.error_word;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(di.sms < kCounters ? di.sms : kCounters));
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, kv, d)) return e;
  if (!d.may_split) return cudaSuccess;
  cfg.gridDim = dim3(unsigned(di.sms * 4));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the join always follows programmatically
  return cudaLaunchKernelEx(&cfg, paged_prefill_join_kernel<D>, d, a.heads);
}

template <int D, bool FP8>
cudaError_t launch(const DeviceInfo& di, const PagedKv& kv, const PagedAttnArgs& a,
                   cudaStream_t s, bool pdl) {
  if (a.softcap > kCapSmall) return launch_as<D, FP8, kLargeCap>(di, kv, a, s, pdl);
  if (a.softcap > 0.f || a.slopes || !(a.scale > 0.f))
    return launch_as<D, FP8, kGeneral>(di, kv, a, s, pdl);
  return launch_as<D, FP8, kPlain>(di, kv, a, s, pdl);
}

}  // namespace

size_t paged_prefill_workspace_bytes(int head_dim) {
  // (the decode kernel's counters,) the records of the join, and one part of
  // two row tiles per CTA
  const DeviceInfo* di = device_info();
  const int64_t ctas = di && di->sms < kCounters ? di->sms : kCounters;
  return size_t(kCounters) * 4 + kJoinBytes + size_t(ctas) * 2 * kRows * (head_dim + 2) * 4;
}

cudaError_t launch_paged_prefill(const PagedKv& kv, int head_dim, bool fp8,
                                 const PagedAttnArgs& a, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  if (head_dim == 64)
    return fp8 ? launch<64, true>(*di, kv, a, s, pdl) : launch<64, false>(*di, kv, a, s, pdl);
  return fp8 ? launch<128, true>(*di, kv, a, s, pdl) : launch<128, false>(*di, kv, a, s, pdl);
}

}  // namespace tt

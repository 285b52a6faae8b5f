// The bookkeeping of a drafted step: the masks and positions of its trees,
// the walk that accepts drafts, and the accepted rows moved together.
//
//   mask(i) = bit i | mask(parent(i));  position(i) = past + depth(i)
//   walk: 0, then from i the lowest child c with draft[c] = chosen[i]
//   keep: row past + path[j] -> past + j, for all layers, kv heads, k and v
//
// All three are a few dependent loads and a few KB to a few MB of rows: bound
// by latency.  A sequence's tree is held by one CTA (masks) or one warp (walk).
//
// Measured (the three together, back to back in a graph): one tree of 8 nodes, 24
// layers of 4 kv heads of 128, 6.9 us; 64 trees of up to 32 nodes, 24 layers of 8 kv
// heads of 64 in FP8, 9.4 us.  A launch each, and two to four dependent loads.
#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kTreeThreads = 256;
constexpr int kTreeMost = 32 * kMaxMaskWords;  // nodes that masks can name

// First flat token of sequence b (b = batch: the end), brought into [0, tokens].
__device__ __forceinline__ int64_t start_of(const int32_t* starts, int b, int64_t tokens) {
  const int64_t s = __ldcg(starts + b);
  return s < 0 ? 0 : s > tokens ? tokens : s;
}

// A CTA per sequence, a thread per node, which climbs to the root: the
// parents' numbers fall, so a climb ends.
__global__ void __launch_bounds__(kTreeThreads)
    draft_tree_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ starts,
                      const int32_t* __restrict__ lens, int64_t tokens, int words,
                      uint32_t* __restrict__ masks, int32_t* __restrict__ positions,
                      int32_t* err) {
  __shared__ int up[kTreeMost];
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int64_t s0 = start_of(starts, b, tokens), s1 = start_of(starts, b + 1, tokens);
  const int64_t n = s1 - s0;
  if (n <= 0) return;
  const int most = 32 * words, nodes = n < most ? int(n) : most;
  if (n > most && tid == 0) flag_error(err, kErrShape);
  for (int i = tid; i < nodes; i += kTreeThreads) {
    int p = __ldcg(parents + s0 + i);
    if (p < -1 || p >= i) {
      flag_error(err, kErrShape);
      p = -1;
    }
    up[i] = p;
  }
  __syncthreads();
  const uint32_t past = uint32_t(__ldcg(lens + b)) - uint32_t(n);
  for (int64_t i = tid; i < n; i += kTreeThreads) {
    uint32_t m[kMaxMaskWords] = {};
    uint32_t depth = 0;
    if (i < nodes) {
      for (int at = int(i); at >= 0; at = up[at]) {
#pragma unroll
        for (int w = 0; w < kMaxMaskWords; ++w) m[w] |= (at >> 5) == w ? 1u << (at & 31) : 0u;
        ++depth;
      }
      --depth;
    }
#pragma unroll
    for (int w = 0; w < kMaxMaskWords; ++w)
      if (w < words) masks[(s0 + i) * words + w] = m[w];
    positions[s0 + i] = int32_t(past + depth);
  }
}

// A warp per sequence: the children of a node are looked for by all lanes.
constexpr int kWalkWarps = 4;
__global__ void __launch_bounds__(32 * kWalkWarps)
    draft_accept_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ drafts,
                        const int32_t* __restrict__ chosen, const int32_t* __restrict__ starts,
                        int batch, int64_t tokens, int width, int32_t* __restrict__ path,
                        int32_t* __restrict__ counts, int32_t* __restrict__ next) {
  const int lane = threadIdx.x & 31, b = blockIdx.x * kWalkWarps + (threadIdx.x >> 5);
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  if (b >= batch) return;
  const int64_t s0 = start_of(starts, b, tokens), s1 = start_of(starts, b + 1, tokens);
  const int n = s1 > s0 ? int(s1 - s0) : 0;
  // the first nodes' parents, drafts and chosen tokens: one round trip
  constexpr int kHeld = 4;
  int up[kHeld], own[kHeld], pick[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const int i = 32 * e + lane;
    up[e] = i < n ? __ldcg(parents + s0 + i) : -1;
    own[e] = i < n ? __ldcg(drafts + s0 + i) : 0;
    pick[e] = i < n ? __ldcg(chosen + s0 + i) : 0;
  }
  auto chosen_of = [&](int i) {
    int v = 0;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) v = (i >> 5) == e ? pick[e] : v;
    v = __shfl_sync(kAll, v, i & 31);
    return i < 32 * kHeld ? v : __ldcg(chosen + s0 + i);
  };
  int32_t* out = path + int64_t(b) * width;
  int count = 0, at = n > 0 ? 0 : -1, last = -1;
  while (at >= 0 && count < width) {
    if (lane == 0) out[count] = at;
    ++count;
    const int want = chosen_of(at);
    last = want;
    int found = -1;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int i = 32 * e + lane;
      const uint32_t hit = __ballot_sync(kAll, i > at && i < n && up[e] == at && own[e] == want);
      if (found < 0 && hit) found = 32 * e + __ffs(hit) - 1;
    }
    for (int i0 = 32 * kHeld; found < 0 && i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const bool yes = i > at && i < n && __ldcg(parents + s0 + i) == at &&
                       __ldcg(drafts + s0 + i) == want;
      const uint32_t hit = __ballot_sync(kAll, yes);
      if (hit) found = i0 + __ffs(hit) - 1;
    }
    at = found;
  }
  for (int j = count + lane; j < width; j += 32) out[j] = -1;
  if (lane == 0) {
    counts[b] = count;
    next[b] = last;
  }
}

// What a sequence keeps, checked: `past`, and the length of the path as far as it
// is one (ascending numbers of new tokens).  By a whole warp.
struct Kept {
  int past, count;
};
__device__ __forceinline__ Kept kept_of(const PagedKv& kv, const int32_t* starts,
                                        const int32_t* path, int width, const int32_t* counts,
                                        int b, int lane, int32_t* err) {
  const int s0 = max(__ldcg(starts + b), 0), s1 = __ldcg(starts + b + 1);
  const int n = s1 > s0 ? s1 - s0 : 0;
  const int most = n < width ? n : width;
  int count = __ldcg(counts + b);
  if (count < 0 || count > most) {
    if (lane == 0) flag_error(err, kErrShape);
    count = count < 0 ? 0 : most;
  }
  const int32_t* p = path + int64_t(b) * width;
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int j = j0 + lane;
    bool bad = false;
    if (j < count) {
      const int at = __ldcg(p + j), before = j > 0 ? __ldcg(p + j - 1) : -1;
      bad = at <= before || at >= n || at < 0;
    }
    const uint32_t hit = __ballot_sync(kAll, bad);
    if (hit) {
      if (lane == 0) flag_error(err, kErrShape);
      count = j0 + __ffs(hit) - 1;
    }
  }
  return {paged_len(kv, b, err) - n, count};
}

// A share of one sequence's columns (16-byte pieces of the rows, and scales) a
// CTA, a column a thread, which moves it for all kept rows in order.  A path
// ascends, so a row is written only after it was read: path[j] >= j, and where it
// is j nothing moves.
constexpr int kKeepThreads = 256;
constexpr int kKeepRows = 256;  // moves looked up at a time
constexpr int kInFlight = 8;
template <bool kScales>
__device__ __forceinline__ void move_rows(const int2* moves, int n, uint8_t* base, int64_t row_bytes,
                                          int64_t head_rows) {
  using T = typename std::conditional<kScales, float, uint4>::type;
  for (int i0 = 0; i0 < n; i0 += kInFlight) {
    T x[kInFlight];
#pragma unroll
    for (int e = 0; e < kInFlight; ++e)
      if (i0 + e < n)
        x[e] = __ldcg(reinterpret_cast<const T*>(base + (moves[i0 + e].x + head_rows) * row_bytes));
#pragma unroll
    for (int e = 0; e < kInFlight; ++e)
      if (i0 + e < n)
        *reinterpret_cast<T*>(base + (moves[i0 + e].y + head_rows) * row_bytes) = x[e];
  }
}

template <int kRow, bool FP8>  // bytes of a cache row
__global__ void __launch_bounds__(kKeepThreads)
    paged_keep_kernel(const PagedKv kv, const __grid_constant__ PagedPools pools,
                      const int32_t* __restrict__ starts, const int32_t* __restrict__ path,
                      int width, const int32_t* __restrict__ counts, int32_t* lens_out,
                      int32_t* err) {
  __shared__ int2 moves[kKeepRows];
  __shared__ int s_past, s_count, s_moves;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  if (tid < 32) {
    const Kept k = kept_of(kv, starts, path, width, counts, b, lane, blockIdx.x == 0 ? err : nullptr);
    if (lane == 0) {
      s_past = k.past;
      s_count = k.count;
      if (lens_out && blockIdx.x == 0) lens_out[b] = max(k.past + k.count, 0);
    }
  }
  __syncthreads();
  const int past = s_past, count = s_count;
  constexpr int kPieces = kRow / 16;
  const int cols = pools.layers * 2 * kv.kv_heads * kPieces;
  const int scales = FP8 ? pools.layers * 2 * kv.kv_heads : 0;
  for (int j0 = 0; j0 < count; j0 += kKeepRows) {
    if (tid == 0) s_moves = 0;
    __syncthreads();
    // the moves of these rows, in order: one warp, so that the order is the path's
    if (tid < 32) {
      int n = 0;
      for (int j1 = j0; j1 < count && j1 < j0 + kKeepRows; j1 += 32) {
        const int j = j1 + lane;
        int src = -1, dst = -1;
        if (j < count && j < j0 + kKeepRows) {
          const int at = __ldcg(path + int64_t(b) * width + j);
          const int t0 = past + at, t1 = past + j;
          if (at != j && t1 >= 0) {
            const int p0 = paged_page(kv, b, t0, err), p1 = paged_page(kv, b, t1, err);
            if (p0 >= 0 && p1 >= 0) {
              src = int(paged_row(kv, p0, 0, t0));
              dst = int(paged_row(kv, p1, 0, t1));
            }
          }
        }
        const uint32_t have = __ballot_sync(kAll, src >= 0);
        if (src >= 0) moves[n + __popc(have & ((1u << lane) - 1u))] = make_int2(src, dst);
        n += __popc(have);
      }
      if (lane == 0) s_moves = n;
    }
    __syncthreads();
    const int n = s_moves;
    if (n > 0) {
      for (int u = blockIdx.x * kKeepThreads + tid; u < cols + scales; u += gridDim.x * kKeepThreads) {
        if (u < cols) {
          const int c = u % kPieces, h = u / kPieces;
          const int j = h % kv.kv_heads, l = h / kv.kv_heads;
          uint8_t* base = static_cast<uint8_t*>(l & 1 ? pools.v[l >> 1] : pools.k[l >> 1]) + 16 * c;
          move_rows<false>(moves, n, base, kRow, int64_t(j) << kv.page_shift);
        } else {
          const int h = u - cols, j = h % kv.kv_heads, l = h / kv.kv_heads;
          float* base = l & 1 ? pools.v_scales[l >> 1] : pools.k_scales[l >> 1];
          move_rows<true>(moves, n, reinterpret_cast<uint8_t*>(base), 4,
                          int64_t(j) << kv.page_shift);
        }
      }
    }
    __syncthreads();
  }
}

// The new lengths, where they go over the old ones: behind the kernel above, whose
// CTAs read those.
__global__ void __launch_bounds__(32 * kWalkWarps)
    keep_lens_kernel(const PagedKv kv, const int32_t* __restrict__ starts,
                     const int32_t* __restrict__ path, int width,
                     const int32_t* __restrict__ counts, int32_t* lens_out) {
  const int lane = threadIdx.x & 31, b = blockIdx.x * kWalkWarps + (threadIdx.x >> 5);
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  if (b >= kv.batch) return;
  const Kept k = kept_of(kv, starts, path, width, counts, b, lane, nullptr);
  if (lane == 0) lens_out[b] = max(k.past + k.count, 0);
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(dim3 grid, int threads, cudaStream_t s, bool pdl) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
  }
};

}  // namespace

cudaError_t launch_draft_tree(const int32_t* parents, const int32_t* starts, const int32_t* lens,
                              int batch, int64_t tokens, int words, uint32_t* masks,
                              int32_t* positions, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  Launch l(dim3(unsigned(batch)), kTreeThreads, s, pdl);
  return cudaLaunchKernelEx(&l.cfg, draft_tree_kernel, parents, starts, lens, tokens, words, masks,
                            positions, di->error_word);
}

cudaError_t launch_draft_accept(const int32_t* parents, const int32_t* drafts,
                                const int32_t* chosen, const int32_t* starts, int batch,
                                int64_t tokens, int width, int32_t* path, int32_t* counts,
                                int32_t* next, cudaStream_t s, bool pdl) {
  Launch l(dim3(unsigned((batch + kWalkWarps - 1) / kWalkWarps)), 32 * kWalkWarps, s, pdl);
  return cudaLaunchKernelEx(&l.cfg, draft_accept_kernel, parents, drafts, chosen, starts, batch,
                            tokens, width, path, counts, next);
}

cudaError_t launch_paged_keep(const PagedKv& kv, const PagedPools& pools, int head_dim, bool fp8,
                              const int32_t* starts, const int32_t* path, int width,
                              const int32_t* counts, int32_t* lens_out, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  auto kern = head_dim == 64 ? (fp8 ? paged_keep_kernel<64, true> : paged_keep_kernel<128, false>)
                             : (fp8 ? paged_keep_kernel<128, true> : paged_keep_kernel<256, false>);
  const int units = pools.layers * 2 * kv.kv_heads * (head_dim * (fp8 ? 1 : 2) / 16 + (fp8 ? 1 : 0));
  const int slices = (units + kKeepThreads - 1) / kKeepThreads;
  const bool over = lens_out == kv.lens;
  Launch l(dim3(unsigned(slices), unsigned(kv.batch)), kKeepThreads, s, pdl);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, kv, pools, starts, path, width, counts,
                                         over ? static_cast<int32_t*>(nullptr) : lens_out,
                                         di->error_word))
    return e;
  if (!over) return cudaSuccess;
  Launch m(dim3(unsigned((kv.batch + kWalkWarps - 1) / kWalkWarps)), 32 * kWalkWarps, s, true);
  return cudaLaunchKernelEx(&m.cfg, keep_lens_kernel, kv, starts, path, width, counts, lens_out);
}

}  // namespace tt

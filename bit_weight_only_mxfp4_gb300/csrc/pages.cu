// Pages of the paged cache: taken and let go (resize), shared and copied (fork),
// moved together (compact).
//
// Which pages are free is read off the table each time: a page is in use if some
// entry names it (or others hold it).  So there are no counts that could go
// wrong, and the order in which free pages are taken, lowest first, does not
// depend on what ran before.
//
// Plan, one CTA: the table's entries set bits (of shared memory, or of the
// workspace where the pool has more pages than that holds), a scan over the words
// gives every free page its number, a scan over the sequences says who gets
// which.  A fork marks the pages that sequences end inside of last: one that is marked
// by then is named elsewhere, and nobody may go on in it.  Copy, all SMs: a warp per
// (page, layer, k or v, kv head) moves the rows, 16 bytes a lane.  The plan is latency
// (a few scans and round trips; the table streams through one SM), the copy is bytes.
//
// Measured (back to back in a graph).  Fork and resize: 4 beams of up to 1000 tokens, 36
// layers of 4 kv heads of 128, 10.2 us; 128 sequences, 24 layers of 8 kv heads of 64 in
// FP8, 71 MB read and written, 27.5 us (single launches from cold caches: the copy 13.7, a
// plan 8.5).  Compaction: 2.5 GB read and written in 402 us (6.2 TB/s, 0.92 of the rate of
// a copy).
#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kErrSize = 8;  // TT_ERR_SIZE
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSharedWords = 40 * 1024;  // bits of 1.3 million pages
constexpr int kHead = 256;               // bytes of the workspace's first part

// The workspace.
struct Space {
  int32_t* head;   // [0] copies
  int4* copies;    // from page, to page, rows
  int32_t* list;   // pages by number: free ones; of a compaction, where a page goes
  uint32_t* bits;  // where shared memory does not hold them
  int32_t* rows;   // the new table, until it may replace the old one
};
struct SpaceSizes {
  int64_t copies, list, bits, rows;
};
inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
SpaceSizes space_sizes(int64_t pages, int64_t batch, int64_t width) {
  const int64_t copies = batch > pages / 2 ? batch : pages / 2;
  return {up16(copies * 16), up16(pages * 4), up16((pages + 31) / 32 * 4), up16(batch * width * 4)};
}
Space space_of(void* ws, int64_t pages, int64_t batch, int64_t width) {
  const SpaceSizes z = space_sizes(pages, batch, width);
  uint8_t* p = static_cast<uint8_t*>(ws);
  Space s;
  s.head = reinterpret_cast<int32_t*>(p);
  s.copies = reinterpret_cast<int4*>(p + kHead);
  s.list = reinterpret_cast<int32_t*>(p + kHead + z.copies);
  s.bits = reinterpret_cast<uint32_t*>(p + kHead + z.copies + z.list);
  s.rows = reinterpret_cast<int32_t*>(p + kHead + z.copies + z.list + z.bits);
  return s;
}

// Sum over the threads before this one; the total in `all`.  `part`: [kWarps + 1].
__device__ __forceinline__ int scan(int v, int* part, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kAll, run, o);
    if (lane >= o) run += u;
  }
  if (lane == 31) part[warp] = run;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w - own;
    if (lane == 31) part[kWarps] = w;
  }
  __syncthreads();
  all = part[kWarps];
  const int before = part[warp] + run - v;
  __syncthreads();
  return before;
}

// Word w's pages that exist and are not held.
__device__ __forceinline__ uint32_t open_pages(const uint8_t* held, int w, int pages) {
  const int p0 = w * 32, n = pages - p0;
  uint32_t m = n >= 32 ? kAll : n <= 0 ? 0u : (1u << n) - 1u;
  if (held) {
    for (int i = 0; i < 32 && i < n; ++i)
      if (__ldcg(held + p0 + i)) m &= ~(1u << i);
  }
  return m;
}

// The first `need` free pages into list, in order; returns how many are free.
__device__ __forceinline__ int free_pages(const uint32_t* bits, const uint8_t* held, int pages,
                                          int need, int32_t* list, int* part) {
  const int words = (pages + 31) / 32, per = (words + kThreads - 1) / kThreads;
  const int w0 = threadIdx.x * per;
  int n = 0;
  for (int w = w0; w < w0 + per && w < words; ++w) n += __popc(open_pages(held, w, pages) & ~bits[w]);
  int all;
  int at = scan(n, part, all);
  for (int w = w0; w < w0 + per && w < words && at < need; ++w) {
    uint32_t m = open_pages(held, w, pages) & ~bits[w];
    for (; m && at < need; m &= m - 1u) list[at++] = w * 32 + __ffs(m) - 1;
  }
  __syncthreads();
  return all;
}

__device__ __forceinline__ void clear(uint32_t* bits, int pages) {
  for (int w = threadIdx.x; w < (pages + 31) / 32; w += kThreads) bits[w] = 0u;
}

// An entry of the table as it is used: a page, or -1; marks the page.
__device__ __forceinline__ void mark(uint32_t* bits, int p, int pages, int32_t* err) {
  if (p >= pages) flag_error(err, kErrShape);
  if (p >= 0 && p < pages) atomicOr(bits + (p >> 5), 1u << (p & 31));
}

// The warps of the CTA shared out among the rows of the table: `team` warps a row.
struct Team {
  int row, rows, lane, lanes;  // first row and step; first entry and step
};
__device__ __forceinline__ Team team_of(int batch) {
  int team = 1;
  while (team < kWarps && batch * team * 2 <= kWarps) team *= 2;
  const int warp = threadIdx.x >> 5;
  return {warp / team, kWarps / team, (warp % team) * 32 + int(threadIdx.x & 31), team * 32};
}

// Pages that sequences end inside of and would write on.  The other entries' pages are
// marked; these are marked here, and those of several threads listed in `twice` (room for
// one a thread).  Whether `page` (of this thread; -1: none) was marked before.  By all
// threads.
__device__ __forceinline__ bool named_before(uint32_t* bits, int page, int* twice, int* count) {
  const uint32_t bit = 1u << (page & 31);
  if (threadIdx.x == 0) *count = 0;
  const bool named = page >= 0 && (bits[page >> 5] & bit);
  __syncthreads();
  if (page >= 0 && !named && (atomicOr(bits + (page >> 5), bit) & bit))
    twice[atomicAdd(count, 1)] = page;
  __syncthreads();
  return named;
}
__device__ __forceinline__ bool is_twice(int page, const int* twice, const int* count) {
  bool more = false;
  for (int i = 0; i < *count; ++i) more |= twice[i] == page;
  return more;
}
// Whether another entry names the thread's page.
__device__ __forceinline__ bool shares_page(uint32_t* bits, int page, int* twice, int* count) {
  return named_before(bits, page, twice, count) || (page >= 0 && is_twice(page, twice, count));
}
// Whether the thread's sequence keeps its page: the first one of those that stay, else the
// first one, unless another entry names it.  `first`: it is the first of those that come
// from one source; ends, sources [batch].
__device__ __forceinline__ bool keeps_page(uint32_t* bits, int page, bool first, int* ends,
                                           const int* sources, int batch, int* twice, int* count) {
  const int tid = threadIdx.x;
  if (!first) page = -1;
  if (tid < batch) ends[tid] = page;
  bool keeps = !named_before(bits, page, twice, count) && page >= 0;
  if (keeps && is_twice(page, twice, count)) {
    const bool stays = sources[tid] == tid;
    for (int i = 0; i < batch; ++i) {
      const bool other = sources[i] == i;
      if (ends[i] == page && (other != stays ? other : i < tid)) keeps = false;
    }
  }
  return keeps;
}

extern __shared__ uint32_t s_bits[];

__global__ void __launch_bounds__(kThreads, 1)
    resize_kernel(const PagedKv kv, const int32_t* want, const uint8_t* held, int32_t* table_out,
                  int32_t* lens_out, int32_t* left, Space ws, bool shared, int32_t* err) {
  __shared__ int part[kWarps + 1];
  __shared__ int count[kPagedMaxBatch], from[kPagedMaxBatch], upto[kPagedMaxBatch];
  __shared__ int s_twice;
  uint32_t* bits = shared ? s_bits : ws.bits;
  const int tid = threadIdx.x, lane = tid & 31, W = kv.pages_per_seq, page = 1 << kv.page_shift;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  clear(bits, kv.num_pages);
  int cut_page = -1;
  if (tid < kv.batch) {
    int w = __ldcg(want + tid);
    const int len = paged_len(kv, tid, err);
    if (w > W << kv.page_shift) {
      flag_error(err, kErrShape);
      w = W << kv.page_shift;
    }
    count[tid] = 0;
    from[tid] = w < 0 ? W : (len + page - 1) >> kv.page_shift;
    upto[tid] = w < 0 ? W : (w + page - 1) >> kv.page_shift;
    lens_out[tid] = w < 0 || w > len ? len : w;
    if (w >= 0 && w < len && (w & (page - 1)) != 0) {
      cut_page = __ldcg(kv.page_table + int64_t(tid) * W + (w >> kv.page_shift));
      if (cut_page >= kv.num_pages) cut_page = -1;
    }
    if (cut_page >= 0) from[tid] = W + 1;  // (no entry is taken)
  }
  const bool cuts = __syncthreads_or(cut_page >= 0);
  const Team t = team_of(kv.batch);
  for (int b = t.row; b < kv.batch; b += t.rows) {
    const int64_t row = int64_t(b) * W;
    const int first = from[b], need = upto[b];
    int missing = 0;
    for (int e0 = t.lane; e0 < W; e0 += 4 * t.lanes) {
      int p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = e0 + i * t.lanes < W ? __ldcg(kv.page_table + row + e0 + i * t.lanes) : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i * t.lanes;
        if (e >= W) break;
        if (e < need) {
          mark(bits, p[i], kv.num_pages, err);
          if (e >= first && (p[i] < 0 || p[i] >= kv.num_pages)) {
            p[i] = -1;
            ++missing;
          }
        } else {
          p[i] = -1;
        }
        table_out[row + e] = p[i];
      }
    }
    missing = __reduce_add_sync(kAll, missing);
    if (lane == 0 && missing) atomicAdd(&count[b], missing);
  }
  __syncthreads();
  if (cuts) {  // the marks again, but for the pages that sequences are cut inside of
    clear(bits, kv.num_pages);
    __syncthreads();
    for (int b = t.row; b < kv.batch; b += t.rows)
      for (int e = t.lane; e < upto[b]; e += t.lanes)
        if (from[b] <= W || e + 1 < upto[b])
          mark(bits, table_out[int64_t(b) * W + e], kv.num_pages, nullptr);
    __syncthreads();
    if (shares_page(bits, cut_page, reinterpret_cast<int*>(ws.copies), &s_twice))
      flag_error(err, kErrSize);
  }
  int all;
  const int mine = tid < kv.batch ? count[tid] : 0;
  const int before = scan(mine, part, all);
  const int have = free_pages(bits, held, kv.num_pages, all, ws.list, part);
  if (tid < kv.batch) count[tid] = mine ? before : -1;
  if (tid == 0) {
    if (left) *left = have - all;
    if (have < all) flag_error(err, kErrSize);
  }
  __syncthreads();
  for (int b = tid >> 5; b < kv.batch; b += kWarps) {
    int at = count[b];
    if (at < 0) continue;
    for (int e0 = from[b]; e0 < upto[b]; e0 += 32) {
      const int e = e0 + lane;
      int32_t* entry = table_out + int64_t(b) * W + e;
      const bool miss = e < upto[b] && *entry < 0;
      const uint32_t hit = __ballot_sync(kAll, miss);
      const int i = at + __popc(hit & ((1u << lane) - 1u));
      if (miss && i < have) *entry = ws.list[i];
      at += __popc(hit);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const PagedKv kv, const int32_t* from, const uint8_t* held, int32_t* table_out,
                int32_t* lens_out, int32_t* left, Space ws, bool shared, int32_t* err) {
  __shared__ int part[kWarps + 1];
  __shared__ int owner[kPagedMaxBatch], source[kPagedMaxBatch], upto[kPagedMaxBatch];
  __shared__ int tail[kPagedMaxBatch];
  __shared__ int s_twice;
  uint32_t* bits = shared ? s_bits : ws.bits;
  const int tid = threadIdx.x, W = kv.pages_per_seq, page = 1 << kv.page_shift;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  clear(bits, kv.num_pages);
  int src = -1, len = 0;
  if (tid < kv.batch) {
    src = __ldcg(from + tid);
    if (src >= kv.batch) {
      flag_error(err, kErrShape);
      src = tid;
    }
    if (src >= 0) len = paged_len(kv, src, err);
    owner[tid] = kPagedMaxBatch;
  }
  __syncthreads();
  // who comes first of a source's: the source if it stays, else its first copy
  if (src >= 0) atomicMin(&owner[src], src == tid ? -1 : tid);
  int old = -1;  // the page that the sequence ends inside of
  if (tid < kv.batch) {
    const int last = len >> kv.page_shift;
    if (src >= 0 && (len & (page - 1)) != 0) {
      old = __ldcg(kv.page_table + int64_t(src) * W + last);
      if (old >= kv.num_pages) old = -1;
    }
    source[tid] = src;
    upto[tid] = src < 0 ? 0 : src == tid ? W : (len + page - 1) >> kv.page_shift;
    tail[tid] = old >= 0 ? last : -1;
  }
  __syncthreads();
  if (tid < kv.batch) lens_out[tid] = len;
  int32_t* rows = table_out == kv.page_table ? ws.rows : table_out;
  const Team t = team_of(kv.batch);
  for (int b = t.row; b < kv.batch; b += t.rows) {
    const int64_t to = int64_t(b) * W, at = int64_t(max(source[b], 0)) * W;
    const int need = upto[b], skip = tail[b];
    for (int e0 = t.lane; e0 < W; e0 += 4 * t.lanes) {
      int p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i * t.lanes;
        p[i] = e < need && e != skip ? __ldcg(kv.page_table + at + e) : -1;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i * t.lanes;
        if (e >= W) break;
        mark(bits, p[i], kv.num_pages, err);
        rows[to + e] = p[i];
      }
    }
  }
  __syncthreads();
  const bool first = src >= 0 && owner[src] == (src == tid ? -1 : tid);
  const bool keeps = keeps_page(bits, old, first, upto, source, kv.batch,
                                reinterpret_cast<int*>(ws.copies), &s_twice);
  const bool copies = old >= 0 && !keeps;
  int all;
  const int at = scan(copies ? 1 : 0, part, all);
  const int have = free_pages(bits, held, kv.num_pages, all, ws.list, part);
  if (keeps) rows[int64_t(tid) * W + tail[tid]] = old;
  if (copies && at < have) {
    const int to = ws.list[at];
    rows[int64_t(tid) * W + tail[tid]] = to;
    ws.copies[at] = make_int4(old, to, len & (page - 1), 0);
  }
  if (tid == 0) {
    ws.head[0] = all < have ? all : have;
    if (left) *left = have - all;
    if (have < all) flag_error(err, kErrSize);
  }
  if (rows == table_out) return;
  __syncthreads();
  for (int64_t i = tid; i < int64_t(kv.batch) * W; i += kThreads) table_out[i] = rows[i];
}

__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(const PagedKv kv, const uint8_t* held, int32_t* table_out, int32_t* span,
                   Space ws, bool shared, int32_t* err) {
  __shared__ int part[kWarps + 1];
  __shared__ int s_end;
  uint32_t* bits = shared ? s_bits : ws.bits;
  const int tid = threadIdx.x, W = kv.pages_per_seq, pages = kv.num_pages;
  const int64_t entries = int64_t(kv.batch) * W;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  clear(bits, pages);
  if (tid == 0) s_end = 0;
  __syncthreads();
  for (int64_t i0 = tid; i0 < entries; i0 += 4 * kThreads) {
    int p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = i0 + i * kThreads < entries ? __ldcg(kv.page_table + i0 + i * kThreads) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) mark(bits, p[i], pages, err);
  }
  __syncthreads();
  // numbers of a page among the open ones, and of a used one among the used
  const int words = (pages + 31) / 32, per = (words + kThreads - 1) / kThreads;
  const int w0 = tid * per;
  int open = 0, used = 0;
  for (int w = w0; w < w0 + per && w < words; ++w) {
    const uint32_t o = open_pages(held, w, pages);
    open += __popc(o);
    used += __popc(o & bits[w]);
  }
  int all_open, all_used;
  const int open0 = scan(open, part, all_open), used0 = scan(used, part, all_used);
  // the place behind the first all_used open pages
  for (int w = w0, at = open0; w < w0 + per && w < words; ++w) {
    uint32_t o = open_pages(held, w, pages);
    const int n = __popc(o);
    if (at < all_used && all_used <= at + n) {
      for (int i = all_used - at; i > 1; --i) o &= o - 1u;
      s_end = w * 32 + __ffs(o);
    }
    at += n;
  }
  __syncthreads();
  const int end = s_end;
  // used ones below it
  auto below = [&](int w, uint32_t m) {
    const int n = end - w * 32;
    return n <= 0 ? 0u : n >= 32 ? m : m & ((1u << n) - 1u);
  };
  int low = 0;
  for (int w = w0; w < w0 + per && w < words; ++w)
    low += __popc(below(w, open_pages(held, w, pages) & bits[w]));
  int all_low;
  (void)scan(low, part, all_low);
  const int moves = all_used - all_low;
  int o_at = open0, u_at = used0;
  for (int w = w0; w < w0 + per && w < words; ++w) {
    const uint32_t o = open_pages(held, w, pages), u = o & bits[w];
    uint32_t hole = below(w, o & ~u);
    for (; hole; hole &= hole - 1u) {
      const int i = __ffs(hole) - 1;
      const uint32_t under = (1u << i) - 1u;
      ws.copies[o_at + __popc(o & under) - u_at - __popc(u & under)].y = w * 32 + i;
    }
    uint32_t goes = u & ~below(w, kAll);
    for (; goes; goes &= goes - 1u) {
      const int i = __ffs(goes) - 1;
      ws.copies[u_at + __popc(u & ((1u << i) - 1u)) - all_low].x = w * 32 + i;
    }
    o_at += __popc(o);
    u_at += __popc(u);
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kThreads) {
    const int4 c = ws.copies[i];
    ws.copies[i].z = 1 << kv.page_shift;
    ws.list[c.x] = c.y;
  }
  if (tid == 0) {
    ws.head[0] = moves;
    if (span) *span = end;
  }
  __syncthreads();
  for (int64_t i = tid; i < entries; i += kThreads) {
    int p = __ldcg(kv.page_table + i);
    if (p >= end && p < pages && !(held && __ldcg(held + p))) p = ws.list[p];
    table_out[i] = p;
  }
}

// The copies of a plan, in every layer: a warp per (copy, layer, k or v, kv head).
// No page is both read and written: a fork reads pages in use and writes free ones,
// a compaction reads past the end and writes before it.
constexpr int kCopyThreads = 256;
constexpr int kInFlight = 8;
template <int kRow, bool FP8>  // bytes of a cache row
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const __grid_constant__ PagedPools pools, int kv_heads, int page_shift,
                      const int32_t* head, const int4* copies) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();
  const int per = pools.layers * 2 * kv_heads;
  const int64_t units = int64_t(__ldcg(head)) * per;
  const int64_t step = int64_t(gridDim.x) * (kCopyThreads / 32);
  for (int64_t u = int64_t(blockIdx.x) * (kCopyThreads / 32) + warp; u < units; u += step) {
    const int i = int(u / per), r = int(u % per);
    const int j = r % kv_heads, l = r / kv_heads;
    const int4 c = __ldcg(copies + i);
    const int64_t src = (int64_t(c.x) * kv_heads + j) << page_shift;
    const int64_t dst = (int64_t(c.y) * kv_heads + j) << page_shift;
    uint8_t* base = static_cast<uint8_t*>(l & 1 ? pools.v[l >> 1] : pools.k[l >> 1]);
    const uint4* from = reinterpret_cast<const uint4*>(base + src * kRow);
    uint4* to = reinterpret_cast<uint4*>(base + dst * kRow);
    const int n = c.z * (kRow / 16);
    for (int p0 = lane; p0 < n; p0 += 32 * kInFlight) {
      uint4 x[kInFlight];
#pragma unroll
      for (int e = 0; e < kInFlight; ++e)
        if (p0 + 32 * e < n) x[e] = __ldcs(from + p0 + 32 * e);
#pragma unroll
      for (int e = 0; e < kInFlight; ++e)
        if (p0 + 32 * e < n) __stcs(to + p0 + 32 * e, x[e]);
    }
    if constexpr (FP8) {
      float* s = l & 1 ? pools.v_scales[l >> 1] : pools.k_scales[l >> 1];
      for (int p = lane; p < c.z; p += 32) s[dst + p] = __ldcg(s + src + p);
    }
  }
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(unsigned grid, int threads, int smem, cudaStream_t s, bool pdl) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
  }
};

// Bytes of shared memory for the bits (0: they lie in the workspace).
int bit_bytes(const PagedKv& kv) {
  const int words = (kv.num_pages + 31) / 32;
  return words <= kSharedWords ? words * 4 : 0;
}

cudaError_t copy_pages(const DeviceInfo& di, const PagedKv& kv, const PagedPools& pools,
                       int head_dim, bool fp8, const Space& ws, int64_t most, cudaStream_t s) {
  auto kern = head_dim == 64 ? (fp8 ? copy_pages_kernel<64, true> : copy_pages_kernel<128, false>)
                             : (fp8 ? copy_pages_kernel<128, true> : copy_pages_kernel<256, false>);
  const int64_t warps = most * pools.layers * 2 * kv.kv_heads;
  const int64_t ctas = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const int64_t full = int64_t(di.sms) * (2048 / kCopyThreads);
  Launch l(unsigned(ctas < full ? ctas : full), kCopyThreads, 0, s, true);
  return cudaLaunchKernelEx(&l.cfg, kern, pools, kv.kv_heads, kv.page_shift,
                            static_cast<const int32_t*>(ws.head), static_cast<const int4*>(ws.copies));
}

}  // namespace

size_t paged_pages_workspace_bytes(int64_t num_pages, int64_t batch, int64_t pages_per_seq) {
  const SpaceSizes z = space_sizes(num_pages, batch, pages_per_seq);
  return size_t(kHead + z.copies + z.list + z.bits + z.rows);
}

cudaError_t launch_paged_resize(const PagedKv& kv, const int32_t* want, const uint8_t* held,
                                int32_t* table_out, int32_t* lens_out, int32_t* left, void* ws,
                                cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  const int smem = bit_bytes(kv);
  if (cudaError_t e = ensure_smem(*di, resize_kernel, smem)) return e;
  Launch l(1, kThreads, smem, s, pdl);
  return cudaLaunchKernelEx(&l.cfg, resize_kernel, kv, want, held, table_out, lens_out, left,
                            space_of(ws, kv.num_pages, kv.batch, kv.pages_per_seq), smem > 0,
                            di->error_word);
}

cudaError_t launch_paged_fork(const PagedKv& kv, const PagedPools& pools, int head_dim, bool fp8,
                              const int32_t* from, const uint8_t* held, int32_t* table_out,
                              int32_t* lens_out, int32_t* left, void* ws, cudaStream_t s,
                              bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  const int smem = bit_bytes(kv);
  if (cudaError_t e = ensure_smem(*di, fork_kernel, smem)) return e;
  const Space space = space_of(ws, kv.num_pages, kv.batch, kv.pages_per_seq);
  Launch l(1, kThreads, smem, s, pdl);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, fork_kernel, kv, from, held, table_out, lens_out,
                                         left, space, smem > 0, di->error_word))
    return e;
  return copy_pages(*di, kv, pools, head_dim, fp8, space, kv.batch, s);
}

cudaError_t launch_paged_compact(const PagedKv& kv, const PagedPools& pools, int head_dim,
                                 bool fp8, const uint8_t* held, int32_t* table_out, int32_t* span,
                                 void* ws, cudaStream_t s, bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  const int smem = bit_bytes(kv);
  if (cudaError_t e = ensure_smem(*di, compact_kernel, smem)) return e;
  const Space space = space_of(ws, kv.num_pages, kv.batch, kv.pages_per_seq);
  Launch l(1, kThreads, smem, s, pdl);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, compact_kernel, kv, held, table_out, span, space,
                                         smem > 0, di->error_word))
    return e;
  const int64_t most = kv.num_pages / 2;
  return copy_pages(*di, kv, pools, head_dim, fp8, space, most < 1 ? 1 : most, s);
}

}  // namespace tt

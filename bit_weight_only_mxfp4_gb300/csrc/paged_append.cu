// Appending a step's keys and values to the paged cache, with the position
// rotation of queries and keys on the way.
//
//   pair i of a head: elements (i, i + rot/2), or (2i, 2i + 1) interleaved
//   a = position[axis(i)] * inv_freq[i]
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a);  dims >= rot pass
//   q -> q_out (bf16);  k, v -> the token's row of the cache, in bf16 or as
//   E4M3 codes with the row's scale amax / 448 (values and scale from the
//   unrounded rotated row).
//
// Angles.  A frequency is kept as a fixed-point fraction of a turn,
// F = round(inv_freq / 2 pi * 2^64), so position * F mod 2^64 is the phase in
// units of 2^-64 turn: one integer product, exact, whatever the position
// (fp32 angles are off by 0.03 rad at position 10^6).  Its top 32 bits go to
// sincospi, rounded to 2^-24 of the half turn.
//
// Bound by bytes for a prompt (every row read and written once) and by
// latency for a decode step.  A CTA takes one or two tokens: its threads look
// up the tokens' places and compute each sine and cosine once, into shared
// memory, and after one barrier each group of head_dim/16 lanes rotates one
// row at a time, a lane both elements of its eight pairs (two 16-byte pieces),
// with the next rows' loads in flight.
//
// Measured (back to back in a graph): one token of 16 / 4 heads of 128 2.1 us,
// 64 tokens of 64 / 8 heads of 64 into FP8 3.0 us, a launch's latency and three
// dependent loads.  Prompts: 6484 tokens of 28 / 4 heads of 128, three axes,
// 23.6 us (5.1 TB/s, waits for loads); 8191 tokens of 40 / 10 heads of 128 into
// FP8 42.5 us (5.4 TB/s; issue slots 70% busy, the 16 divisions of a lane's
// part of a row weigh most: a quotient has to be the nearest one, or codes
// that lie between two others would differ from the quantiser's).  Two rows' loads
// in flight instead of one: 23.9 / 46.0 us; at most 40 registers a thread for
// more CTAs: 23.9 / 48.4.
#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

constexpr int kThreads = 128;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int64_t kNowhere = INT64_MIN;  // the place of a token that no sequence has

__global__ void rope_turns_kernel(const double* __restrict__ inv_freq, int n,
                                  uint64_t* __restrict__ turns) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  // the fraction of a turn in [0, 1): whole turns move nothing
  const double t = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
  const double s = rint((t - floor(t)) * 18446744073709551616.0);  // 2^64
  turns[i] = s >= 18446744073709551616.0 ? 0ull : uint64_t(s);
}

struct AppendArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, kv_stride;
  const int32_t* starts;
  int heads;
  RopeArgs rope;
  uint16_t* q_out;
  int32_t* err;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Two E4M3 codes, a's in the low byte: nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// kTok tokens per CTA; blockIdx.y: a share of their rows.
template <int D, bool FP8, int kTok>
__global__ void __launch_bounds__(kThreads)
    paged_append_kernel(const PagedKv kv, const AppendArgs a, int64_t tokens) {
  constexpr int U = D / 16;            // lanes per row
  constexpr int RPC = kThreads / U;    // rows per round
  constexpr int kPairs = D / 2;
  __shared__ float2 cs[kTok][kPairs];  // pair 8u + k at [k * U + u]: lanes read side by side
  __shared__ int s_page[kTok];
  __shared__ int64_t s_place[kTok];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t t0 = int64_t(blockIdx.x) * kTok;
  const int unit = tid % U;
  const int rows = a.heads + 2 * kv.kv_heads;
  const int rot = a.rope.turns ? a.rope.rot : 0;
  // this lane's two pieces of 8 elements: the elements of its pairs, or two
  // neighbours past the rotated part
  const bool turns = unit < rot / 16;
  const bool halved = turns && !a.rope.interleaved;
  const int p0 = halved ? unit : 2 * unit;
  const int p1 = halved ? unit + rot / 16 : 2 * unit + 1;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();

  struct Two {
    uint4 x, y;
  };
  auto source = [&](int tk, int r) {
    const int64_t t = t0 + tk;
    const uint16_t* p = r < a.heads ? a.q + t * a.q_stride + int64_t(r) * D
                        : r < a.heads + kv.kv_heads
                            ? a.k + t * a.kv_stride + int64_t(r - a.heads) * D
                            : a.v + t * a.kv_stride + int64_t(r - a.heads - kv.kv_heads) * D;
    const uint4* u = reinterpret_cast<const uint4*>(p);
    return Two{__ldcg(u + p0), __ldcg(u + p1)};
  };
  // this thread's rows: (token, row), RPC rows further each round
  int tk = 0, r = blockIdx.y * RPC + tid / U;
  const int step = gridDim.y * RPC;
  const int ntok = tokens - t0 < kTok ? int(tokens - t0) : kTok;
  auto settle = [&] {
    while (r >= rows && tk < ntok) {
      r -= rows;
      ++tk;
    }
  };
  settle();
  Two raw{};
  if (tk < ntok) raw = source(tk, r);

  // ---- places and angles: one pair of one token a thread
  constexpr int kShare = kThreads / kTok < kPairs ? kThreads / kTok : kPairs;
  if (tid < kTok * kShare) {
    const int my = tid / kShare;  // a warp has one token
    const int64_t t = t0 + my;
    if (my < ntok) {
      const bool says = tid % kShare == 0;
      int32_t* e = says ? a.err : nullptr;
      int b = int(t);
      int64_t place;
      if (a.starts && kv.batch < 32) {
        // all starts and lengths in one round trip
        const int s = lane <= kv.batch ? __ldcg(a.starts + lane) : INT32_MAX;
        const int n = lane < kv.batch ? paged_len(kv, lane, a.err) : 0;
        b = __popc(__ballot_sync(kAll, lane > 0 && lane < kv.batch && s <= t));
        const int s0 = __shfl_sync(kAll, s, b), s1 = __shfl_sync(kAll, s, b + 1);
        const int len = __shfl_sync(kAll, n, b);
        place = t >= s0 && t < s1 ? len - (s1 - t) : kNowhere;
      } else if (a.starts) {
        b = paged_seq_of(a.starts, kv.batch, t, lane);
        const int64_t s0 = __ldcg(a.starts + b), s1 = __ldcg(a.starts + b + 1);
        const int n = paged_len(kv, b, e);
        place = t >= s0 && t < s1 ? n - (s1 - t) : kNowhere;
      } else {
        place = int64_t(paged_len(kv, b, e)) - 1;
      }
      if (says) {
        s_place[my] = place;
        s_page[my] = place >= 0 ? paged_page(kv, b, place, e) : -1;
      }
      for (int i = tid % kShare; i < rot / 2; i += kShare) {
        int64_t pos = place;
        if (a.rope.positions) {
          int ax = a.rope.pair_axis ? a.rope.pair_axis[i] : 0;
          ax = ax < a.rope.axes ? ax : a.rope.axes - 1;
          pos = __ldcg(a.rope.positions + int64_t(ax) * tokens + t);
        }
        const uint64_t ph = uint64_t(pos) * a.rope.turns[i];
        float sn, cn;
        sincospif(float(int32_t(ph >> 32)) * 0x1p-31f, &sn, &cn);
        cs[my][(i & 7) * U + (i >> 3)] = make_float2(cn, sn);
      }
    }
  }
  __syncthreads();

  // ---- rows: the whole warp stays while any of its lanes has one
  while (__any_sync(kAll, tk < ntok)) {
    const bool have = tk < ntok;
    const int ct = have ? tk : 0, cr = r;
    float x[8], y[8];
    unpack8(raw.x, x);
    unpack8(raw.y, y);
    r += step;
    settle();
    if (tk < ntok) raw = source(tk, r);
    const bool is_v = cr >= a.heads + kv.kv_heads;
    if (turns && !is_v) {
      if (halved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 c = cs[ct][k * U + unit];
          const float u = x[k] * c.x - y[k] * c.y;
          y[k] = x[k] * c.y + y[k] * c.x;
          x[k] = u;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 c = cs[ct][k * U + unit];
          float* z = k < 4 ? x + 2 * k : y + 2 * (k - 4);
          const float u = z[0] * c.x - z[1] * c.y;
          z[1] = z[0] * c.y + z[1] * c.x;
          z[0] = u;
        }
      }
    }
    const int64_t place = s_place[ct];
    const int page = s_page[ct];
    if (have && cr < a.heads && place != kNowhere) {
      const bool in = place >= 0;
      uint4* o = reinterpret_cast<uint4*>(a.q_out + ((t0 + ct) * a.heads + cr) * D);
      o[p0] = in ? pack8(x) : make_uint4(0u, 0u, 0u, 0u);
      o[p1] = in ? pack8(y) : make_uint4(0u, 0u, 0u, 0u);
    }
    const bool store = have && cr >= a.heads && page >= 0 && place >= 0;
    const int j = cr - a.heads - (is_v ? kv.kv_heads : 0);
    const int64_t row = store ? paged_row(kv, page, j, place) : 0;
    if constexpr (FP8) {
      if (!__any_sync(kAll, store)) continue;  // a warp of query rows
      // a NaN or an infinity gives the row a NaN scale and zero codes
      float m = 0.f, z = 0.f;  // z: 0, or NaN if any element is not finite
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m = fmaxf(m, fmaxf(fabsf(x[k]), fabsf(y[k])));
        z = fmaf(x[k], 0.f, fmaf(y[k], 0.f, z));
      }
      if (!(z == 0.f)) m = INFINITY;
#pragma unroll
      for (int o = U / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      if (store) {
        const bool ok = m < INFINITY;
        const float s = m / 448.f;
        uint32_t c[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        if (ok && s > 0.f) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            c[k] = e4m3x2(x[2 * k] / s, x[2 * k + 1] / s);
            c[k + 4] = e4m3x2(y[2 * k] / s, y[2 * k + 1] / s);
          }
        }
        uint2* o = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? kv.v : kv.k) + row * D);
        o[p0] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        o[p1] = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
        if (unit == 0)
          (is_v ? kv.v_scales : kv.k_scales)[row] = ok ? s : __int_as_float(0x7fc00000);
      }
    } else if (store) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? kv.v : kv.k) + row * D);
      o[p0] = pack8(x);
      o[p1] = pack8(y);
    }
  }
}

template <int D, bool FP8>
cudaError_t launch(const DeviceInfo& di, const PagedKv& kv, const AppendArgs& a, int64_t tokens,
                   cudaStream_t s, bool pdl) {
  const int per = kThreads / (D / 16);
  const int rounds = (a.heads + 2 * kv.kv_heads + per - 1) / per;
  // Few tokens (a decode step): a CTA per token and round of rows, so that no
  // row waits for another.  From eight tokens per SM on, two tokens a CTA, which
  // goes through all of their rows: 128 threads and 2 tokens took 23.6 / 42.5 us
  // on the bf16 / FP8 prompts of 6484 / 8191 tokens, 256 and 4 24.6 / 48.1, 512
  // and 8 25.9 / 49.2.
  const bool many = tokens >= 8 * di.sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = many ? dim3(unsigned((tokens + 1) / 2)) : dim3(unsigned(tokens), unsigned(rounds));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return many ? cudaLaunchKernelEx(&cfg, paged_append_kernel<D, FP8, 2>, kv, a, tokens)
              : cudaLaunchKernelEx(&cfg, paged_append_kernel<D, FP8, 1>, kv, a, tokens);
}

}  // namespace

cudaError_t launch_rope_turns(const double* inv_freq, int n, uint64_t* turns, cudaStream_t s) {
  rope_turns_kernel<<<(n + 127) / 128, 128, 0, s>>>(inv_freq, n, turns);
  return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedKv& kv, int head_dim, bool fp8, const uint16_t* q,
                                const uint16_t* k, const uint16_t* v, int64_t q_stride,
                                int64_t kv_stride, int64_t tokens, const int32_t* starts,
                                int heads, const RopeArgs& rope, uint16_t* q_out, cudaStream_t s,
                                bool pdl) {
  const DeviceInfo* di = device_info();
  if (!di) return cudaErrorNoDevice;
  const AppendArgs a{q, k, v, q_stride, kv_stride, starts, heads, rope, q_out, di->error_word};
  if (head_dim == 64)
    return fp8 ? launch<64, true>(*di, kv, a, tokens, s, pdl)
               : launch<64, false>(*di, kv, a, tokens, s, pdl);
  return fp8 ? launch<128, true>(*di, kv, a, tokens, s, pdl)
             : launch<128, false>(*di, kv, a, tokens, s, pdl);
}

}  // namespace tt

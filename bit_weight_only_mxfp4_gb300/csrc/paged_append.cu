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
// latency for a decode step.  A CTA takes one token and a share of its
// heads: it computes the rot/2 sines and cosines once into shared memory
// while its first rows of q, k and v are already on their way, and each
// group of head_dim/8 lanes then rotates one row: 16 bytes a lane, the
// partner elements by shuffle.
#include "launch.h"
#include "paged.cuh"

namespace tt {
namespace {

constexpr int kThreads = 256;
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

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    paged_append_kernel(const PagedKv kv, const AppendArgs a) {
  constexpr int LPR = D / 8;           // lanes per row
  constexpr int RPC = kThreads / LPR;  // rows per CTA and round
  __shared__ float2 cs[D / 2];
  __shared__ int s_page;
  __shared__ int64_t s_place;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t t = blockIdx.x;
  const int sub = tid % LPR;
  const int rows = a.heads + 2 * kv.kv_heads;
  const int rot = a.rope.turns ? a.rope.rot : 0, half = rot >> 1;
  pdl_allow_next_grid();
  pdl_wait_prior_grid();

  auto source = [&](int r) {
    const uint16_t* p = r < a.heads ? a.q + t * a.q_stride + int64_t(r) * D
                        : r < a.heads + kv.kv_heads
                            ? a.k + t * a.kv_stride + int64_t(r - a.heads) * D
                            : a.v + t * a.kv_stride + int64_t(r - a.heads - kv.kv_heads) * D;
    return __ldcg(reinterpret_cast<const uint4*>(p) + sub);
  };
  int r = blockIdx.y * RPC + tid / LPR;
  uint4 raw = r < rows ? source(r) : make_uint4(0u, 0u, 0u, 0u);

  // Warp 0: the token's sequence, place and page.
  if (tid < 32) {
    const int b = a.starts ? paged_seq_of(a.starts, kv.batch, t, lane) : int(t);
    int32_t* e = lane == 0 ? a.err : nullptr;
    const int len = paged_len(kv, b, e);
    int64_t place = int64_t(len) - 1;
    if (a.starts) {
      const int64_t s0 = __ldcg(a.starts + b), s1 = __ldcg(a.starts + b + 1);
      place = t >= s0 && t < s1 ? len - (s1 - t) : kNowhere;
    }
    const int page = place >= 0 ? paged_page(kv, b, place, e) : -1;
    if (lane == 0) {
      s_page = page;
      s_place = place;
    }
  }
  __syncthreads();
  const int64_t place = s_place;
  const int page = s_page;
  if (place == kNowhere) return;
  for (int i = tid; i < half; i += kThreads) {
    int64_t pos = place;
    if (a.rope.positions) {
      int ax = a.rope.pair_axis ? a.rope.pair_axis[i] : 0;
      ax = ax < a.rope.axes ? ax : a.rope.axes - 1;
      pos = __ldcg(a.rope.positions + int64_t(ax) * gridDim.x + t);
    }
    const uint64_t ph = uint64_t(pos) * a.rope.turns[i];
    float sn, cn;
    sincospif(float(int32_t(ph >> 32)) * 0x1p-31f, &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();

  const int step = gridDim.y * RPC;
  for (; r - tid / LPR < rows; r += step) {
    const uint4 next = r + step < rows ? source(r + step) : make_uint4(0u, 0u, 0u, 0u);
    float x[8];
    unpack8(raw, x);
    if (rot) {
      float y[8];
      if (a.rope.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = 8 * sub < rot ? cs[4 * sub + i] : make_float2(1.f, 0.f);
          y[2 * i] = x[2 * i] * c.x - x[2 * i + 1] * c.y;
          y[2 * i + 1] = x[2 * i] * c.y + x[2 * i + 1] * c.x;
        }
      } else {
        const int hl = half >> 3;  // lanes of the first half
        const bool first = sub < hl, in = 8 * sub < rot;
        const int from = !in ? lane : first ? lane + hl : lane - hl;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(kAll, x[i], from);
          const float2 c = in ? cs[8 * (first ? sub : sub - hl) + i] : make_float2(1.f, 0.f);
          y[i] = x[i] * c.x + (first ? -o : o) * c.y;
          if (!in) y[i] = x[i];
        }
      }
      if (8 * sub < rot && r < a.heads + kv.kv_heads) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i];
      }
    }
    if (r < a.heads) {
      const uint4 w = place >= 0 ? pack8(x) : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(a.q_out + (t * a.heads + r) * D + 8 * sub) = w;
    }
    const int jr = r - a.heads;  // k head, or kv_heads + v head
    const bool is_k = jr < kv.kv_heads;
    const int j = is_k ? jr : jr - kv.kv_heads;
    const bool store = jr >= 0 && r < rows && page >= 0;
    const int64_t row = store ? paged_row(kv, page, j, place) : 0;
    if constexpr (FP8) {
      // a NaN or an infinity gives the row a NaN scale and zero codes
      float m = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(x[i]));
        bad |= !(fabsf(x[i]) <= 3.4028234663852886e38f);
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      const uint32_t votes = __ballot_sync(kAll, bad);
      const uint32_t row_lanes = ((1u << LPR) - 1) << (lane & ~(LPR - 1));
      if (store) {
        const bool ok = (votes & row_lanes) == 0u;
        const float s = m / 448.f;
        uint32_t c[4] = {0u, 0u, 0u, 0u};
        if (ok && s > 0.f) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x[2 * i] / s, x[2 * i + 1] / s);
        }
        uint8_t* base = static_cast<uint8_t*>(is_k ? kv.k : kv.v);
        *reinterpret_cast<uint2*>(base + row * D + 8 * sub) =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        if (sub == 0)
          (is_k ? kv.k_scales : kv.v_scales)[row] = ok ? s : __int_as_float(0x7fc00000);
      }
    } else if (store) {
      uint16_t* base = static_cast<uint16_t*>(is_k ? kv.k : kv.v);
      *reinterpret_cast<uint4*>(base + row * D + 8 * sub) = pack8(x);
    }
    raw = next;
  }
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
  const int per = kThreads / (head_dim / 8);
  const int rounds = (heads + 2 * kv.kv_heads + per - 1) / per;
  // Few tokens: a CTA per round of rows, so that no row waits for another;
  // many: one CTA goes through all of a token's rows on one set of angles.
  const int share = tokens * rounds <= 4 * di->sms ? rounds : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tokens), unsigned(share));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (head_dim == 64)
    return fp8 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<64, true>, kv, a)
               : cudaLaunchKernelEx(&cfg, paged_append_kernel<64, false>, kv, a);
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<128, true>, kv, a)
             : cudaLaunchKernelEx(&cfg, paged_append_kernel<128, false>, kv, a);
}

}  // namespace tt

// RMSNorm of each q and k head, rotation by the position, and the write to the paged cache.
//
// Every element is read once and written once (k and v into the cache), so the bound is memory:
// 4 bytes an element in 16-bit types.
//
// Angles: theta is needed modulo one turn only.  inv_freq / (2 pi) is held as a 64-bit
// fixed-point fraction of a turn, and position * fraction wraps modulo 2^64 by itself, so one
// integer product reduces exactly; the top 32 bits, as a signed fraction of a turn, go to
// sincospi.  The fraction's error is below 2^-53 of its value (the binary64 product) plus
// 2^-64, so at position 2^20 and one radian a position the angle is off by less than 2^-35 turns,
// under the 2^-33 of the cut to 32 bits.
#include "ar_common.cuh"
#include "ar_serve.h"

namespace ar {
namespace {

constexpr int kRopeThreads = 256;

// Fraction of a turn a position, in units of 2^-64 turns (modulo 1).
__device__ __forceinline__ unsigned long long turn_of(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return (unsigned long long)(t * 18446744073709549568.0);  // t < 1; 2^64 less one ulp keeps it in range
}

__device__ __forceinline__ void angle(unsigned long long turn, int pos, float* s, float* c) {
  const unsigned long long a = turn * (unsigned long long)(long long)pos;
  const int top = (int)(unsigned)((a + 0x80000000ull) >> 32);  // [-0.5, 0.5) turns in units of 2^-32
  sincospif((float)top * 0x1p-31f, s, c);                      // 2 pi turns = pi * (2 turns)
}

// The position axis of frequency i.
__device__ __forceinline__ int axis_of(const RopeParams& p, int i) {
  if (p.axes == 1) return 0;
  if (!p.dealt) {
    int a = 0;
    for (int end = p.sections[0]; a < p.axes - 1 && i >= end;) end += p.sections[++a];
    return a;
  }
  // round k deals one frequency to each axis whose section is longer than k
  int left = i;
  for (int k = 0; k <= i; ++k)
    for (int a = 0; a < p.axes; ++a)
      if (k < p.sections[a] && left-- == 0) return a;
  return 0;
}

// Any alignment, stride and head size: one warp a head, its values as fp32 in shared memory.
template <int DT>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar(const __grid_constant__ RopeParams p) {
  __shared__ float buf[kRopeThreads / 32][AR_MAX_HEAD_DIM];
  pdl_wait_and_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.q.heads + p.k.heads * (p.k_cache ? 2 : 1);
  const int64_t total = p.tokens * heads;
  float* x = buf[warp];
  for (int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + warp; w < total; w += (int64_t)gridDim.x * (kRopeThreads / 32)) {
    const int64_t t = w / heads;
    int h = (int)(w - t * heads);
    const bool is_q = h < p.q.heads, is_v = h >= p.q.heads + p.k.heads;
    int64_t slot = -1;
    if (!is_q && p.k_cache) {
      slot = p.slots[t];
      if (slot < -1 || slot >= p.num_slots) {
        slot = -1;
        if (lane == 0) *p.status = kStatusBadIndex;
      }
    }
    const int64_t blk = slot < 0 ? 0 : slot / p.page, off = slot < 0 ? 0 : slot - blk * p.page;
    if (is_v) {
      h -= p.q.heads + p.k.heads;
      if (slot < 0) continue;
      const uint16_t* src = static_cast<const uint16_t*>(p.v) + t * p.v_ts + h * p.v_hs;
      uint16_t* dst = static_cast<uint16_t*>(p.v_cache) + blk * p.vc_bs + off * p.vc_ps + h * p.vc_hs;
      for (int e = lane; e < p.head_dim; e += 32) st_u16(dst + e, ld_u16(src + e));
      continue;
    }
    const HeadRows& r = is_q ? p.q : p.k;
    if (!is_q) h -= p.q.heads;
    const uint16_t* src = static_cast<const uint16_t*>(r.in) + t * r.in_ts + h * r.in_hs;
    float ss = 0.0f;
    for (int e = lane; e < p.head_dim; e += 32) {
      unsigned short b;  // a plain load: the output may be this very row
      asm volatile("ld.global.u16 %0, [%1];" : "=h"(b) : "l"(src + e) : "memory");
      x[e] = to_f32<DT>(b);
      ss += x[e] * x[e];
    }
    if (r.weight) {
      const float rs = rsqrtf(warp_sum(ss) * p.inv_dim + p.eps);
      for (int e = lane; e < p.head_dim; e += 32) {
        const float wt = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(r.weight) + e));
        x[e] = x[e] * rs * (p.gemma ? 1.0f + wt : wt);
      }
    }
    __syncwarp();
    for (int i = lane; i < p.half; i += 32) {
      float s, c;
      angle(turn_of(p.inv_freq[i]), p.positions[axis_of(p, i) * p.pos_stride + t], &s, &c);
      const int ia = p.pairs ? 2 * i : i, ib = p.pairs ? 2 * i + 1 : i + p.half;
      const float a = x[ia], b = x[ib];
      x[ia] = a * c - b * s;
      x[ib] = b * c + a * s;
    }
    __syncwarp();
    uint16_t* dst = r.out ? static_cast<uint16_t*>(r.out) + t * r.out_ts + h * r.out_hs : nullptr;
    uint16_t* dc = slot < 0 ? nullptr : static_cast<uint16_t*>(p.k_cache) + blk * p.kc_bs + off * p.kc_ps + h * p.kc_hs;
    for (int e = lane; e < p.head_dim; e += 32) {
      const uint16_t y = round1<DT>(x[e]);
      if (dst) st_u16(dst + e, y);
      if (dc) st_u16(dc + e, y);
    }
    __syncwarp();
  }
}

// 16-byte load that an in-place store may follow: coherent, and not moved across it.
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kMaxTokensPerStep = 4;
constexpr int kHeadsInFlight = 4;
enum RopeMode { kPairs = 0, kHalves8 = 1, kHalvesAny = 2 };

// Rows on 16-byte boundaries and heads of a multiple of 8 elements: L lanes hold a head, 8
// elements each (L the power of two at or above head_dim / 8), so a warp serves 32 / L heads at
// a time.  A CTA takes `step` tokens: it computes their angles once, for all heads, into shared
// memory (a sincos a head would cost more than the memory traffic does), and each lane keeps
// the eight that its elements need in registers over the heads of a token.  Four heads a
// lane are loaded before the first is worked on, so that an SM has about 48 KB in flight.  The
// partner of an element is in the lane itself (pairs), in one other lane at the same place
// (halves that are a multiple of 8: a shuffle), or anywhere (kHalvesAny: through shared
// memory, rows of 8 skewed by one float so that lanes fall into different banks).
// With few tokens the heads are shared out over `split` CTAs a token.
template <int DT, int L, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_vec(const __grid_constant__ RopeParams p, int step, int split) {
  constexpr int GROUPS = kRopeThreads / L;
  __shared__ unsigned long long turn[AR_MAX_HEAD_DIM / 2];
  __shared__ int axis[AR_MAX_HEAD_DIM / 2];
  __shared__ __align__(16) float cosv[kMaxTokensPerStep][AR_MAX_HEAD_DIM / 2 + 8];
  __shared__ __align__(16) float sinv[kMaxTokensPerStep][AR_MAX_HEAD_DIM / 2 + 8];
  __shared__ int64_t k_at[kMaxTokensPerStep], v_at[kMaxTokensPerStep];  // cache offsets of a token, -1: none
  __shared__ float skew[MODE == kHalvesAny ? kRopeThreads * 9 : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int e0 = lane * 8;
  const bool there = e0 < p.head_dim;
  pdl_wait_and_release();
  for (int i = threadIdx.x; i < p.half; i += kRopeThreads) {
    turn[i] = turn_of(p.inv_freq[i]);
    axis[i] = axis_of(p, i);
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (there && p.q.weight) wq = ld_keep(static_cast<const uint16_t*>(p.q.weight) + e0);
  if (there && p.k.weight) wk = ld_keep(static_cast<const uint16_t*>(p.k.weight) + e0);
  const float one = p.gemma ? 1.0f : 0.0f;
  // the place of this lane's first frequency, and whether its elements turn
  const int f0 = MODE == kPairs ? lane * 4 : (e0 < p.half ? e0 : e0 - p.half);

  const int heads = p.q.heads + p.k.heads * (p.k_cache ? 2 : 1);
  const int per = (heads + split - 1) / split;
  const int64_t units = (p.tokens + step - 1) / step * split;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t t0 = u / split * step;
    const int h_lo = (int)(u % split) * per, h_hi = min(h_lo + per, heads);
    const int n = (int)min((int64_t)step, p.tokens - t0);
    __syncthreads();
    for (int x = threadIdx.x; x < n * p.half; x += kRopeThreads) {
      const int t = x / p.half, i = x - t * p.half;
      angle(turn[i], p.positions[axis[i] * p.pos_stride + t0 + t], &sinv[t][i], &cosv[t][i]);
    }
    if (p.k_cache && threadIdx.x >= kRopeThreads - 32 && (int)threadIdx.x - (kRopeThreads - 32) < n) {
      const int t = threadIdx.x - (kRopeThreads - 32);
      const int64_t slot = p.slots[t0 + t];
      k_at[t] = v_at[t] = -1;
      if (slot >= 0 && slot < p.num_slots) {
        const int64_t b = slot / p.page, off = slot - b * p.page;
        k_at[t] = b * p.kc_bs + off * p.kc_ps;
        v_at[t] = b * p.vc_bs + off * p.vc_ps;
      } else if (slot != -1) {
        *p.status = kStatusBadIndex;
      }
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < (MODE == kPairs ? 4 : 8); ++i) {
        const int f = MODE == kHalvesAny ? (e0 + i < p.half ? e0 + i : e0 + i - p.half) : f0 + i;
        const bool turns = MODE == kHalvesAny ? e0 + i < 2 * p.half : f < p.half;
        c[i] = turns ? cosv[t][f] : 0.0f;
        s[i] = turns ? sinv[t][f] : 0.0f;
        if (MODE != kPairs && e0 + i < p.half) s[i] = -s[i];  // a' = a cos - b sin, b' = b cos + a sin
      }
      for (int hb = h_lo + group; hb - group < h_hi; hb += GROUPS * kHeadsInFlight) {
        uint4 raw[kHeadsInFlight];
#pragma unroll
        for (int j = 0; j < kHeadsInFlight; ++j) {
          const int h = hb + j * GROUPS;
          raw[j] = make_uint4(0, 0, 0, 0);
          if (h < h_hi && there) {
            const uint16_t* src;
            if (h < p.q.heads)
              src = static_cast<const uint16_t*>(p.q.in) + (t0 + t) * p.q.in_ts + h * p.q.in_hs;
            else if (h < p.q.heads + p.k.heads)
              src = static_cast<const uint16_t*>(p.k.in) + (t0 + t) * p.k.in_ts + (h - p.q.heads) * p.k.in_hs;
            else
              src = static_cast<const uint16_t*>(p.v) + (t0 + t) * p.v_ts + (h - p.q.heads - p.k.heads) * p.v_hs;
            raw[j] = ld_row(src + e0);
          }
        }
#pragma unroll
        for (int j = 0; j < kHeadsInFlight; ++j) {
          if (hb - group + j * GROUPS >= h_hi) break;  // the same for the whole CTA
          const int h = hb + j * GROUPS;
          const bool is_q = h < p.q.heads, is_v = h >= p.q.heads + p.k.heads;
          float x[8], y[8];
          unpack8<DT>(raw[j], x);
          if (p.q.weight || p.k.weight) {  // the whole warp takes part: its heads may be of different kinds
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (is_q ? p.q.weight != nullptr : p.k.weight != nullptr) {
              const float rs = rsqrtf(ss * p.inv_dim + p.eps);
              float w[8];
              unpack8<DT>(is_q ? wq : wk, w);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * (w[i] + one);
            }
          }
          if constexpr (MODE == kPairs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool turns = f0 + i < p.half;  // an element that does not turn keeps its value, infinities included
              y[2 * i] = turns ? x[2 * i] * c[i] - x[2 * i + 1] * s[i] : x[2 * i];
              y[2 * i + 1] = turns ? x[2 * i + 1] * c[i] + x[2 * i] * s[i] : x[2 * i + 1];
            }
          } else if constexpr (MODE == kHalves8) {
            const int src = e0 < p.half ? lane + p.half / 8 : (e0 < 2 * p.half ? lane - p.half / 8 : lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float other = __shfl_sync(0xffffffffu, x[i], src, L);
              y[i] = e0 < 2 * p.half ? x[i] * c[i] + other * s[i] : x[i];
            }
          } else {
            float* row = skew + group * L * 9;  // element e at e + e / 8
#pragma unroll
            for (int i = 0; i < 8; ++i) row[lane * 9 + i] = x[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = e0 + i, q = e < p.half ? e + p.half : (e < 2 * p.half ? e - p.half : e);
              y[i] = e < 2 * p.half ? x[i] * c[i] + row[q + (q >> 3)] * s[i] : x[i];
            }
            __syncwarp();
          }
          if (h < h_hi && there) {
            if (is_v) {
              if (v_at[t] >= 0) st_v4(static_cast<uint16_t*>(p.v_cache) + v_at[t] + (h - p.q.heads - p.k.heads) * p.vc_hs + e0, raw[j]);
            } else {
              const uint4 out = pack8<DT>(y);
              const HeadRows& r = is_q ? p.q : p.k;
              const int hh = is_q ? h : h - p.q.heads;
              if (r.out) st_v4(static_cast<uint16_t*>(r.out) + (t0 + t) * r.out_ts + hh * r.out_hs + e0, out);
              if (!is_q && p.k_cache && k_at[t] >= 0) st_v4(static_cast<uint16_t*>(p.k_cache) + k_at[t] + hh * p.kc_hs + e0, out);
            }
          }
        }
      }
    }
  }
}

template <int DT, int L>
const void* vec_of(int mode) {
  switch (mode) {
    case kPairs: return reinterpret_cast<const void*>(&rope_vec<DT, L, kPairs>);
    case kHalves8: return reinterpret_cast<const void*>(&rope_vec<DT, L, kHalves8>);
    default: return reinterpret_cast<const void*>(&rope_vec<DT, L, kHalvesAny>);
  }
}

template <int DT>
const void* vec_of(int dim, int mode) {
  if (dim <= 64) return vec_of<DT, 8>(mode);
  return dim <= 128 ? vec_of<DT, 16>(mode) : vec_of<DT, 32>(mode);
}

}  // namespace

const void* rope_scalar_kernel(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&rope_scalar<kBF16>) : reinterpret_cast<const void*>(&rope_scalar<kF16>);
}

const void* rope_vec_kernel(bool bf16, int head_dim, int half, bool pairs) {
  const int mode = pairs ? kPairs : (half % 8 == 0 ? kHalves8 : kHalvesAny);
  return bf16 ? vec_of<kBF16>(head_dim, mode) : vec_of<kF16>(head_dim, mode);
}

RopeGrid rope_vec_grid(const RopeParams& p, int sm_count) {
  // kMaxTokensPerStep tokens a CTA once every resident CTA has one such step, else single
  // tokens; below one token an SM the heads of a token go to several CTAs, as long as each has
  // a round of heads
  const int lanes = p.head_dim <= 64 ? 8 : (p.head_dim <= 128 ? 16 : 32);
  const int heads = p.q.heads + p.k.heads * (p.k_cache ? 2 : 1), groups = kRopeThreads / lanes;
  RopeGrid g;
  g.step = p.tokens >= (int64_t)kMaxTokensPerStep * 3 * sm_count ? kMaxTokensPerStep : 1;
  g.split = 1;
  while (g.step == 1 && p.tokens * g.split < sm_count && heads > groups * g.split) g.split *= 2;
  const int64_t units = (p.tokens + g.step - 1) / g.step * g.split;
  g.ctas = units < (int64_t)3 * sm_count ? (unsigned)units : 3u * sm_count;
  return g;
}

}  // namespace ar

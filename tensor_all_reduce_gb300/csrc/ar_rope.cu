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
#include "ar_fastdiv.cuh"
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

constexpr int kMaxTokensPerStep = 8;
constexpr int kHeadsInFlight = 4;
enum RopeMode { kPairs = 0, kHalves8 = 1, kHalvesAny = 2 };

// a * b, a * b + c on two floats at a time
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Rows on 16-byte boundaries and heads of a multiple of 8 elements: n = head_dim / 8 lanes hold a
// head, 8 elements each, and a warp as many heads as fit (three of 80 elements, for instance;
// LANES = 8, 16 or 32 for the powers of two, where a head's sum is a butterfly, 0 for others).
// A CTA takes `step` tokens: it computes their angles once, for all heads, into shared memory (a
// sincos a head would cost more than the memory traffic does), then works through the tokens' q
// heads, k heads and v heads, four a lane loaded before the first is worked on, so that an SM
// has about 48 KB in flight.  The partner of an element is in the lane itself (pairs), in
// one other lane at the same place (halves that are a multiple of 8: a shuffle), or anywhere
// (kHalvesAny: through shared memory, rows of 8 skewed by one float so that lanes fall into
// different banks).  With few tokens the heads are shared out over `split` CTAs a token.
// Instructions are what bounds it next to memory: offsets within a step are 32-bit, and the
// sine is kept with either sign.
template <int DT, int MODE, int LANES>
struct RopeVec {
  struct Shared {
    unsigned long long turn[AR_MAX_HEAD_DIM / 2];
    int axis[AR_MAX_HEAD_DIM / 2];
    __align__(16) float cosv[kMaxTokensPerStep][AR_MAX_HEAD_DIM / 2 + 8];
    __align__(16) float sinv[2][kMaxTokensPerStep][AR_MAX_HEAD_DIM / 2 + 8];  // -sin, sin
    int64_t k_at[kMaxTokensPerStep], v_at[kMaxTokensPerStep];               // cache offsets of a token, -1: none
    float skew[MODE == kHalvesAny ? kRopeThreads * 9 : 1];
  };

  const RopeParams& p;
  Shared& sh;
  int n, lane, first, group, groups, e0;  // lanes of a head; place in the head; the head's first lane; heads at a time
  bool there;

  __device__ __forceinline__ RopeVec(const RopeParams& params, Shared& shared) : p(params), sh(shared) {
    n = LANES ? LANES : p.head_dim / 8;
    const int per_warp = 32 / n, wl = threadIdx.x & 31, in_warp = wl / n;
    lane = wl - in_warp * n;
    first = in_warp * n;
    there = LANES ? true : in_warp < per_warp;
    groups = per_warp * (kRopeThreads / 32);
    group = (int)(threadIdx.x >> 5) * per_warp + in_warp;
    e0 = lane * 8;
  }

  // Sum over a head's lanes, to all of them.
  __device__ __forceinline__ float head_sum(float s) const {
    if constexpr (LANES != 0) {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s;
    } else {
      // windows of 1, 2, 4, .. lanes by doubling, and the head as the windows that the bits of n
      // name, low bits first
      auto rotated = [&](int by) {
        const int x = lane + by;
        return first + (x >= n ? x - n : x);
      };
      float sum = 0.0f;
      int off = 0;
#pragma unroll
      for (int k = 1; k <= 16; k <<= 1) {
        if (n & k) {
          sum = off ? sum + __shfl_sync(0xffffffffu, s, rotated(off)) : s;
          off += k;
        }
        if (2 * k <= n) s += __shfl_sync(0xffffffffu, s, rotated(k));
      }
      return sum;
    }
  }

  // The q (or k) heads of tokens t0 .. t0 + tokens.
  template <bool KEYS>
  __device__ __forceinline__ void heads(int64_t t0, int tokens, int mine, int stride) {
    const HeadRows& r = KEYS ? p.k : p.q;
    const int total = tokens * r.heads;
    float2 w[4];
    if (r.weight && there) {
      float f[8];
      unpack8<DT>(ld_keep(static_cast<const uint16_t*>(r.weight) + e0), f);
      const float one = p.gemma ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = make_float2(f[2 * i] + one, f[2 * i + 1] + one);
    }
    const uint16_t* in = static_cast<const uint16_t*>(r.in) + t0 * r.in_ts + e0;
    uint16_t* out = r.out ? static_cast<uint16_t*>(r.out) + t0 * r.out_ts + e0 : nullptr;
    const int in_ts = (int)r.in_ts, in_hs = (int)r.in_hs, out_ts = (int)r.out_ts, out_hs = (int)r.out_hs;
    const bool low = e0 < p.half, turns = e0 < 2 * p.half;  // of kHalves8
    const int f0 = turns ? (low ? e0 : e0 - p.half) : 0;
    const int partner = (first + (turns ? (low ? lane + p.half / 8 : lane - p.half / 8) : lane)) & 31;
    for (int base = 0; base < total; base += stride * kHeadsInFlight) {
      uint4 raw[kHeadsInFlight];
#pragma unroll
      for (int j = 0; j < kHeadsInFlight; ++j) {
        const int x = base + j * stride + mine;
        raw[j] = make_uint4(0, 0, 0, 0);
        if (x < total && there) {
          const int t = x / r.div, h = x - t * r.heads;
          raw[j] = ld_row(in + (t * in_ts + h * in_hs));
        }
      }
#pragma unroll
      for (int j = 0; j < kHeadsInFlight; ++j) {
        if (base + j * stride >= total) break;  // the same for the whole CTA
        const int x = base + j * stride + mine;
        const int t = min(x, total - 1) / r.div, h = x - t * r.heads;
        float f[8];
        float2 a[4], y[4];
        unpack8<DT>(raw[j], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = make_float2(f[2 * i], f[2 * i + 1]);
        if (r.weight) {
          float2 ss = mul2(a[0], a[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) ss = fma2(a[i], a[i], ss);
          const float rs = rsqrtf(head_sum(ss.x + ss.y) * p.inv_dim + p.eps);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = mul2(mul2(a[i], make_float2(rs, rs)), w[i]);
        }
        // an element that does not turn keeps its value, infinities included
        if constexpr (MODE == kPairs) {
          const float4 c = *reinterpret_cast<const float4*>(&sh.cosv[t][lane * 4]), s = *reinterpret_cast<const float4*>(&sh.sinv[1][t][lane * 4]);
          const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = a[i];
            if (lane * 4 + i < p.half) y[i] = make_float2(a[i].x * cc[i] - a[i].y * sc[i], a[i].y * cc[i] + a[i].x * sc[i]);
          }
        } else if constexpr (MODE == kHalves8) {
          float2 other[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) other[i] = make_float2(__shfl_sync(0xffffffffu, a[i].x, partner), __shfl_sync(0xffffffffu, a[i].y, partner));
          const float* c = &sh.cosv[t][f0];
          const float* s = &sh.sinv[low ? 0 : 1][t][f0];  // a' = a cos - b sin, b' = b cos + a sin
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float4 c4 = *reinterpret_cast<const float4*>(c + 2 * i), s4 = *reinterpret_cast<const float4*>(s + 2 * i);
            y[i] = a[i];
            y[i + 1] = a[i + 1];
            if (turns) {
              y[i] = fma2(other[i], make_float2(s4.x, s4.y), mul2(a[i], make_float2(c4.x, c4.y)));
              y[i + 1] = fma2(other[i + 1], make_float2(s4.z, s4.w), mul2(a[i + 1], make_float2(c4.z, c4.w)));
            }
          }
        } else {
          float* row = sh.skew + (threadIdx.x - lane) * 9;  // element e at e + e / 8
#pragma unroll
          for (int i = 0; i < 8; ++i) row[lane * 9 + i] = i & 1 ? a[i / 2].y : a[i / 2].x;
          __syncwarp();
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            v[i] = i & 1 ? a[i / 2].y : a[i / 2].x;
            if (there && e < 2 * p.half) {  // (lanes behind the warp's last head would read behind the array)
              const bool lo = e < p.half;
              const int q = lo ? e + p.half : e - p.half, k = lo ? e : q;
              v[i] = v[i] * sh.cosv[t][k] + row[q + (q >> 3)] * sh.sinv[lo ? 0 : 1][t][k];
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = make_float2(v[2 * i], v[2 * i + 1]);
        }
        if (x < total && there) {
          const uint4 z = make_uint4(pack2<DT>(y[0].x, y[0].y), pack2<DT>(y[1].x, y[1].y), pack2<DT>(y[2].x, y[2].y), pack2<DT>(y[3].x, y[3].y));
          if (out) st_v4(out + (t * out_ts + h * out_hs), z);
          if constexpr (KEYS) {
            if (p.k_cache && sh.k_at[t] >= 0) st_v4(static_cast<uint16_t*>(p.k_cache) + sh.k_at[t] + h * p.kc_hs + e0, z);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void values(int64_t t0, int tokens, int mine, int stride) {  // copied
    const int total = tokens * p.k.heads;
    const uint16_t* in = static_cast<const uint16_t*>(p.v) + t0 * p.v_ts + e0;
    const int in_ts = (int)p.v_ts, in_hs = (int)p.v_hs;
    for (int base = 0; base < total; base += stride * kHeadsInFlight) {
      uint4 raw[kHeadsInFlight];
#pragma unroll
      for (int j = 0; j < kHeadsInFlight; ++j) {
        const int x = base + j * stride + mine;
        if (x < total && there) {
          const int t = x / p.k.div, h = x - t * p.k.heads;
          raw[j] = ld_stream(in + (t * in_ts + h * in_hs));
        }
      }
#pragma unroll
      for (int j = 0; j < kHeadsInFlight; ++j) {
        const int x = base + j * stride + mine;
        if (x < total && there) {
          const int t = x / p.k.div, h = x - t * p.k.heads;
          if (sh.v_at[t] >= 0) st_v4(static_cast<uint16_t*>(p.v_cache) + sh.v_at[t] + h * p.vc_hs + e0, raw[j]);
        }
      }
    }
  }

  __device__ __forceinline__ void run(int step, int split) {
    for (int i = threadIdx.x; i < p.half; i += kRopeThreads) {
      sh.turn[i] = turn_of(p.inv_freq[i]);
      sh.axis[i] = axis_of(p, i);
    }
    const int64_t units = (p.tokens + step - 1) / step * split;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
      const int64_t t0 = (split == 1 ? u : u / split) * step;
      const int mine = (split == 1 ? 0 : (int)(u % split) * groups) + group, stride = groups * split;
      const int tokens = (int)min((int64_t)step, p.tokens - t0);
      __syncthreads();
      for (int x = threadIdx.x; x < tokens * p.half; x += kRopeThreads) {
        const int t = x / p.half_div, i = x - t * p.half;
        float s, c;
        angle(sh.turn[i], p.positions[sh.axis[i] * p.pos_stride + t0 + t], &s, &c);
        sh.cosv[t][i] = c;
        sh.sinv[0][t][i] = -s;
        sh.sinv[1][t][i] = s;
      }
      if (p.k_cache && threadIdx.x >= kRopeThreads - 32 && (int)threadIdx.x - (kRopeThreads - 32) < tokens) {
        const int t = threadIdx.x - (kRopeThreads - 32);
        const int64_t slot = p.slots[t0 + t];
        sh.k_at[t] = sh.v_at[t] = -1;
        if (slot >= 0 && slot < p.num_slots) {
          const int64_t b = slot / p.page, off = slot - b * p.page;
          sh.k_at[t] = b * p.kc_bs + off * p.kc_ps;
          sh.v_at[t] = b * p.vc_bs + off * p.vc_ps;
        } else if (slot != -1) {
          *p.status = kStatusBadIndex;
        }
      }
      __syncthreads();
      heads<false>(t0, tokens, mine, stride);
      heads<true>(t0, tokens, mine, stride);
      if (p.k_cache) values(t0, tokens, mine, stride);
    }
  }
};

template <int DT, int MODE, int LANES>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_vec(const __grid_constant__ RopeParams p, int step, int split) {
  __shared__ typename RopeVec<DT, MODE, LANES>::Shared sh;
  pdl_wait_and_release();
  RopeVec<DT, MODE, LANES>(p, sh).run(step, split);
}

template <int DT, int MODE>
const void* vec_of(int dim) {
  switch (dim) {
    case 64: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 8>);
    case 128: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 16>);
    case 256: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 32>);
    default: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 0>);
  }
}

template <int DT>
const void* vec_of(int mode, int dim) {
  return mode == kPairs ? vec_of<DT, kPairs>(dim) : mode == kHalves8 ? vec_of<DT, kHalves8>(dim) : vec_of<DT, kHalvesAny>(dim);
}

}  // namespace

const void* rope_scalar_kernel(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&rope_scalar<kBF16>) : reinterpret_cast<const void*>(&rope_scalar<kF16>);
}

const void* rope_vec_kernel(bool bf16, int head_dim, int half, bool pairs) {
  const int mode = pairs ? kPairs : (half % 8 == 0 ? kHalves8 : kHalvesAny);
  return bf16 ? vec_of<kBF16>(mode, head_dim) : vec_of<kF16>(mode, head_dim);
}

RopeGrid rope_vec_grid(const RopeParams& p, int sm_count) {
  // several tokens a CTA once every resident CTA has such a step, else single tokens; below one
  // token an SM the heads of a token go to several CTAs, as long as each has a round of heads
  const int groups = 32 / (p.head_dim / 8) * (kRopeThreads / 32);
  const int heads = p.q.heads > p.k.heads ? p.q.heads : p.k.heads;
  RopeGrid g;
  g.step = kMaxTokensPerStep;
  while (g.step > 1 && p.tokens < (int64_t)g.step * 3 * sm_count) g.step /= 2;
  g.split = 1;
  while (g.step == 1 && p.tokens * g.split < sm_count && heads > groups * g.split) g.split *= 2;
  const int64_t units = (p.tokens + g.step - 1) / g.step * g.split;
  g.ctas = units < (int64_t)3 * sm_count ? (unsigned)units : 3u * sm_count;
  return g;
}

}  // namespace ar

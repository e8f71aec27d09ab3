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

}  // namespace

const void* rope_kernel(bool bf16, bool vec) {
  (void)vec;
  return bf16 ? reinterpret_cast<const void*>(&rope_scalar<kBF16>) : reinterpret_cast<const void*>(&rope_scalar<kF16>);
}

}  // namespace ar

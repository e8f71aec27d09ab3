// RMSNorm of each q and k head, rotation by the position, and the write to the paged cache.
//
// Every element is read once and written once (k and v into the cache), so the bound is memory:
// 4 bytes an element in 16-bit types.
//
// Angles: theta is needed modulo one turn only.  inv_freq / (2 pi) is held as a 64-bit
// fixed-point fraction of a turn, and position * fraction wraps modulo 2^64 by itself, so one
// integer product reduces exactly; the top 32 bits, as a signed fraction of a turn, go to
// sincospi, which takes 24 of them: 2^-26 turns at most.  The fraction's error is below 2^-52 of
// inv_freq / (2 pi) (the binary64 constant and the product) plus 2^-64, and the position multiplies it: 2^-34
// turns at position 2^20 and one radian a position, as much as the cut at 2^29, 2^-23.6 at 2^31.
#include "ar_common.cuh"
#include "ar_fastdiv.cuh"
#include "ar_serve.h"
#include "ar_staged.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kRopeThreads = 256;   // of the general form
constexpr int kRopeWorkers = 256;   // working threads of the vector form
constexpr int kRopeLoaders = 64;    // and those that run ahead
constexpr int kRopeMaxStep = 8;     // tokens of a unit
constexpr int kRopeRowBytes = 16384;  // a unit of one token has no more heads than this, or one
constexpr int kRopeSmem = 68 * 1024;  // all stages, so that three CTAs fit an SM; kRopeSkew less where halves meet in shared memory
constexpr int kRopeSkew = kRopeWorkers * 18 * 4;
constexpr int kRopeUnitCost = 4096;   // a unit costs as much as so many bytes besides its own

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
  // round k deals one frequency to each axis whose section is longer than k; all rounds up to the
  // end of the shortest section left at once
  int left = i, done = 0;
  for (int phase = 0; phase < p.axes; ++phase) {
    int shortest = 0x7fffffff, open = 0;
    for (int a = 0; a < p.axes; ++a)
      if (p.sections[a] > done) {
        ++open;
        shortest = min(shortest, p.sections[a]);
      }
    if (open == 0) break;
    if (left < (shortest - done) * open) {
      int nth = left % open;
      for (int a = 0; a < p.axes; ++a)
        if (p.sections[a] > done && nth-- == 0) return a;
    }
    left -= (shortest - done) * open;
    done = shortest;
  }
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

constexpr int kStages = 2;  // three of the same size: 2800 and 16384 tokens (below) 24.0, 61.9 us, two 23.3, 60.8
enum RopeMode { kPairs = 0, kHalves8 = 1, kHalvesAny = 2 };

// Rows on 16-byte boundaries and heads of a multiple of 8 elements.  A CTA works through units of
// `step` tokens by `per` heads (q heads, k heads, v heads counted on), staged through a ring in
// shared memory.  Two warps run ahead: one brings the rows in by bulk copies, the other finds the
// tokens' places in the cache, and both compute the units' angles, once for all heads (a sincos
// a head would cost more than the memory traffic does; one warp alone was the bound where rows
// are short).  Eight warps work: n = head_dim / 16 lanes hold a head (rounded up), two chunks of 8
// elements each, and a warp as many heads as fit (six of 80 elements; LANES: n of the usual
// sizes, 0 for others).  The chunks of a lane are chosen so that it has both elements of each
// pair: adjacent pairs anyway, halves of a multiple of 8 as chunk c and the one half a rotation
// on.  Other halves go through shared memory (kHalvesAny; rows of 8 skewed by one float so that
// lanes fall into different banks).
//
// The bound is memory, with the arithmetic not far behind.  Measured on GB300 (CUDA graph, cold
// inputs): 2800 tokens x 64 heads of 128, half rotated, 92 MB: 23.4 us, 3.9 TB/s with the launch (the general form 95 us);
// the same without norm and rotation 18.3 us, without the stores too 13.0 us.  16384 tokens x 48
// heads of 80, adjacent pairs, three axes, 252 MB: 57.0 us, 4.4 TB/s (the general form 600 us).  What it took to get there,
// 2800 and 16384 tokens: rows loaded straight into registers 32 and 89 us; staged 25 and 78 us; two
// chunks a lane instead of shuffles between partners 23 and 70 us; two floats an instruction and
// sums unrolled for n = 5 and 6 24 and 62 us; units of up to 34 KB in two stages 23 and 57 us.
template <int DT, int MODE, int LANES>
struct RopeVec {
  struct Shared {
    uint64_t full[kStages], empty[kStages];
    int64_t k_at[kStages][kRopeMaxStep], v_at[kStages][kRopeMaxStep];  // cache offsets of a token, -1: none
    unsigned long long turn[AR_MAX_HEAD_DIM / 2];
    int axis[AR_MAX_HEAD_DIM / 2];
    __align__(16) float weight[2][AR_MAX_HEAD_DIM];  // w or 1 + w of q and k, in planes
    float skew[MODE == kHalvesAny ? kRopeSkew / 4 : 1];
    int stop;
  };

  const RopeParams& p;
  const RopePlan& plan;
  Shared& sh;
  uint8_t* stage;  // kStages stages: rows, then cosines and sines

  // Eight floats a lane are read as two times 16 bytes.  Neighbouring lanes' 16 bytes stand side by
  // side, so that they fall into different banks: element e of `count` in two planes of four
  // each out of eight.
  __device__ __forceinline__ static int in_planes(int e, int count) { return ((e >> 2) & 1) * (count / 2) + (e >> 3) * 4 + (e & 3); }
  __device__ __forceinline__ int angle_at(int f) const { return MODE == kHalves8 ? in_planes(f, p.half) : f; }

  struct Unit {
    int64_t t0;
    int tokens, lo, hi;  // heads [lo, hi)
  };
  __device__ __forceinline__ Unit unit(int64_t u) const {
    Unit x;
    const int64_t group = plan.split == 1 ? u : u / plan.split;
    x.t0 = group * plan.step;
    x.tokens = (int)min((int64_t)plan.step, p.tokens - x.t0);
    x.lo = (int)(u - group * plan.split) * plan.per;
    x.hi = min(x.lo + plan.per, plan.heads);
    return x;
  }
  __device__ __forceinline__ uint8_t* rows_of(int s) const { return stage + (size_t)s * plan.stage_bytes; }
  __device__ __forceinline__ float* angles_of(int s) const { return reinterpret_cast<float*>(rows_of(s) + plan.row_bytes); }

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
      if (*reinterpret_cast<volatile int*>(&sh.stop)) return false;
      if (clock64() - t0 > p.wait_cycles) {
        *reinterpret_cast<volatile int*>(&sh.stop) = 1;
        *p.status = 1;
        return false;
      }
    }
    return true;
  }

  // Copies the heads [a, b) of one kind that lie in the unit, of token t.
  __device__ __forceinline__ void copy(const Unit& x, int t, int a, int b, const void* in, int64_t ts, int64_t hs, int s) {
    const int lo = max(a, x.lo), hi = min(b, x.hi);
    if (lo >= hi) return;
    const uint32_t head = p.head_dim * 2;
    const uint16_t* src = static_cast<const uint16_t*>(in) + (x.t0 + t) * ts + (lo - a) * hs;
    uint8_t* dst = rows_of(s) + (t * plan.per + lo - x.lo) * head;
    if (hs == p.head_dim) {
      bulk_g2s(dst, src, (hi - lo) * head, &sh.full[s]);
    } else {
      for (int h = lo; h < hi; ++h, src += hs, dst += head) bulk_g2s(dst, src, head, &sh.full[s]);
    }
  }

  __device__ __forceinline__ void load() {
    const int tid = threadIdx.x - kRopeWorkers, lane = tid & 31;
    uint32_t n = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < plan.units; u += gridDim.x, ++n) {
      const int s = n % kStages;
      const Unit x = unit(u);
      ok = __all_sync(0xffffffffu, wait(&sh.empty[s], ((n / kStages) & 1) ^ 1));
      if (!ok) break;
      if (tid < 32) {
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], x.tokens * (x.hi - x.lo) * p.head_dim * 2);
        __syncwarp();
        if (lane < x.tokens * 3 && !(p.stall && n == 0)) {  // a lane a token and kind
          const int t = lane / 3, kind = lane - t * 3;
          if (kind == 0) copy(x, t, 0, p.q.heads, p.q.in, p.q.in_ts, p.q.in_hs, s);
          if (kind == 1) copy(x, t, p.q.heads, p.q.heads + p.k.heads, p.k.in, p.k.in_ts, p.k.in_hs, s);
          if (kind == 2) copy(x, t, p.q.heads + p.k.heads, plan.heads, p.v, p.v_ts, p.v_hs, s);
        }
      } else if (p.k_cache && lane < x.tokens) {
        const int64_t slot = p.slots[x.t0 + lane];
        int64_t k = -1, v = -1;
        if (slot >= 0 && slot < p.num_slots) {
          const int64_t b = slot / p.page, off = slot - b * p.page;
          k = b * p.kc_bs + off * p.kc_ps;
          v = b * p.vc_bs + off * p.vc_ps;
        } else if (slot != -1) {
          *p.status = kStatusBadIndex;
        }
        sh.k_at[s][lane] = k;
        sh.v_at[s][lane] = v;
      }
      float* c = angles_of(s);
      const int size = plan.step * plan.pitch;
#pragma unroll 4
      for (int i = tid; i < x.tokens * p.half; i += kRopeLoaders) {
        const int t = i / p.half_div, f = i - t * p.half;
        float sn, cs;
        angle(sh.turn[f], p.positions[sh.axis[f] * p.pos_stride + x.t0 + t], &sn, &cs);
        const int at = t * plan.pitch + angle_at(f);
        c[at] = cs;
        c[size + at] = sn;
      }
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&sh.full[s])) : "memory");
    }
    if (!ok && tid < 32)  // copies in flight end before the CTA does
      for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
        if (!(p.stall && i == 0)) mbar_wait_bounded(&sh.full[i % kStages], (i / kStages) & 1, p.wait_cycles);
  }

  // Eight floats of chunk c out of two planes, in pairs.
  __device__ __forceinline__ static void planes(const float* p, int plane, int c, uint64_t (&f)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p + c * 4), b = *reinterpret_cast<const ulonglong2*>(p + plane + c * 4);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  }
  __device__ __forceinline__ static void unpack(const uint4& v, uint64_t (&f)[4]) {
    float a[8];
    unpack8<DT>(v, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = two(a[2 * i], a[2 * i + 1]);
  }
  __device__ __forceinline__ static uint4 pack(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      untwo(f[i], a, b);
      w[i] = pack2<DT>(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  __device__ __forceinline__ void work() {
    const int chunks = p.head_dim / 8, n = LANES ? LANES : (chunks + 1) / 2;  // lanes of a head
    const int per_warp = 32 / n, wl = threadIdx.x & 31, in_warp = wl / n;
    const int lane = wl - in_warp * n, first = in_warp * n;  // place in the head; its first lane
    const bool there = 32 % (LANES ? LANES : 32) == 0 && LANES ? true : in_warp < per_warp;
    const int warp = threadIdx.x >> 5;
    // this lane's chunks; `two_chunks`: it has the second
    const int hb = p.half / 8;
    const bool turns = MODE != kHalves8 || lane < hb;
    const int c0 = MODE != kHalves8 || turns ? lane : 2 * lane;
    const int c1_raw = MODE != kHalves8 ? lane + n : (turns ? lane + hb : c0 + 1);
    const bool two_chunks = c1_raw < chunks;
    const int c1 = two_chunks ? c1_raw : c0;
    // Sum over a head's lanes, to all of them.
    auto head_sum = [&](float s) {
      if constexpr (LANES != 0 && (LANES & (LANES - 1)) == 0) {
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
    };
    const int size = plan.step * plan.pitch, head = p.head_dim * 2, v0 = p.q.heads + p.k.heads;
    const int per_round = (kRopeWorkers / 32) * per_warp;
    auto store2 = [&](uint16_t* dst, const uint4& a, const uint4& b) {
      st_v4(dst + c0 * 8, a);
      if (two_chunks) st_v4(dst + c1 * 8, b);
    };
    uint32_t k = 0;
    for (int64_t u = blockIdx.x; u < plan.units; u += gridDim.x, ++k) {
      const int s = k % kStages;
      const Unit x = unit(u);
      const bool ok = wait(&sh.full[s], (k / kStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) return;
      const uint8_t* rows = rows_of(s);
      const float* angles = angles_of(s);
      uint16_t* q_out = static_cast<uint16_t*>(p.q.out) + x.t0 * p.q.out_ts;
      uint16_t* k_out = p.k.out ? static_cast<uint16_t*>(p.k.out) + x.t0 * p.k.out_ts : nullptr;
      const int total = x.tokens * (x.hi - x.lo);
      for (int at = warp * per_warp + in_warp; at - in_warp < total; at += per_round) {
        const bool mine = there && at < total;
        const int i0 = min(at, total - 1);
        const int t = plan.step > 1 ? i0 / plan.heads_div : 0;
        const int h = x.lo + i0 - t * plan.per;
        const uint8_t* row = rows + i0 * head;
        const uint4 raw0 = lds_v4(row + c0 * 16), raw1 = two_chunks ? lds_v4(row + c1 * 16) : make_uint4(0, 0, 0, 0);
        const bool is_q = h < p.q.heads, is_v = h >= v0;
        uint16_t* v_dst = static_cast<uint16_t*>(p.v_cache) + sh.v_at[s][t] + (h - v0) * p.vc_hs;
        if (__all_sync(0xffffffffu, is_v)) {  // v is copied
          if (mine && sh.v_at[s][t] >= 0) store2(v_dst, raw0, raw1);
          continue;
        }
        uint64_t a[4], b[4], y[4], z[4];
        unpack(raw0, a);
        unpack(raw1, b);
        if (p.q.weight || p.k.weight) {
          uint64_t ss = mul2(a[0], a[0]), sb = mul2(b[0], b[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            ss = fma2(a[i], a[i], ss);
            sb = fma2(b[i], b[i], sb);
          }
          float lo, hi;
          untwo(add2(ss, sb), lo, hi);
          const float rs = rsqrtf(head_sum(lo + hi) * p.inv_dim + p.eps);
          if (is_q ? p.q.weight != nullptr : p.k.weight != nullptr) {
            const float* w = sh.weight[is_q ? 0 : 1];
            uint64_t wa[4], wb[4];
            planes(w, p.head_dim / 2, c0, wa);
            planes(w, p.head_dim / 2, c1, wb);
            const uint64_t r2 = two(rs, rs);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = mul2(a[i], mul2(r2, wa[i]));
              b[i] = mul2(b[i], mul2(r2, wb[i]));
            }
          }
        }
        // an element that does not turn keeps its value, infinities included
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = a[i];
          z[i] = b[i];
        }
        const float* c = angles + t * plan.pitch;
        if constexpr (MODE == kPairs) {
          auto turn = [&](int chunk, const uint64_t (&from)[4], uint64_t (&to)[4]) {
            if (chunk * 4 >= p.half) return;
            const float4 c4 = *reinterpret_cast<const float4*>(c + chunk * 4), s4 = *reinterpret_cast<const float4*>(c + size + chunk * 4);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, sc[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (chunk * 4 + i < p.half) {
                float u, v;
                untwo(from[i], u, v);
                to[i] = two(u * cc[i] - v * sc[i], v * cc[i] + u * sc[i]);
              }
          };
          turn(c0, a, y);
          turn(c1, b, z);
        } else if constexpr (MODE == kHalves8) {
          if (turns) {
            uint64_t cc[4], sc[4];
            planes(c, p.half / 2, lane, cc);
            planes(c + size, p.half / 2, lane, sc);
            const uint64_t minus = two(-1.0f, -1.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[i] = fma2(b[i], mul2(sc[i], minus), mul2(a[i], cc[i]));
              z[i] = fma2(a[i], sc[i], mul2(b[i], cc[i]));
            }
          }
        } else {
          float* skew = sh.skew + (threadIdx.x - lane) * 18;  // element e at e + e / 8
          auto write = [&](int chunk, const uint64_t (&from)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) untwo(from[i], skew[chunk * 9 + 2 * i], skew[chunk * 9 + 2 * i + 1]);
          };
          if (there) write(c0, a);  // (lanes behind the warp's last head have no place)
          if (there && two_chunks) write(c1, b);
          __syncwarp();
          auto turn = [&](int chunk, const uint64_t (&from)[4], uint64_t (&to)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[2];
              untwo(from[i], v[0], v[1]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int e = chunk * 8 + 2 * i + j;
                if (there && e < 2 * p.half) {
                  const bool low = e < p.half;
                  const int q = low ? e + p.half : e - p.half, g = low ? e : q;
                  const float other = skew[q + (q >> 3)] * c[size + g];
                  v[j] = v[j] * c[g] + (low ? -other : other);
                }
              }
              to[i] = two(v[0], v[1]);
            }
          };
          turn(c0, a, y);
          turn(c1, b, z);
          __syncwarp();
        }
        if (!mine) continue;
        const uint4 out0 = pack(y), out1 = pack(z);
        if (is_q) {
          store2(q_out + t * p.q.out_ts + h * p.q.out_hs, out0, out1);
        } else if (is_v) {
          if (sh.v_at[s][t] >= 0) store2(v_dst, raw0, raw1);
        } else {
          const int kh = h - p.q.heads;
          if (k_out) store2(k_out + t * p.k.out_ts + kh * p.k.out_hs, out0, out1);
          if (p.k_cache && sh.k_at[s][t] >= 0) store2(static_cast<uint16_t*>(p.k_cache) + sh.k_at[s][t] + kh * p.kc_hs, out0, out1);
        }
      }
      __syncwarp();
      if (wl == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&sh.empty[s])) : "memory");
    }
  }

  __device__ __forceinline__ void run() {
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&sh.full[s], 1 + kRopeLoaders);  // the copies' bytes, and each loading thread
        mbar_init(&sh.empty[s], kRopeWorkers / 32);
      }
      sh.stop = 0;
      mbar_fence_init();
      fence_proxy_async_smem();
    }
    pdl_wait_and_release();
    for (int i = threadIdx.x; i < p.half; i += kRopeWorkers + kRopeLoaders) {
      sh.turn[i] = turn_of(p.inv_freq[i]);
      sh.axis[i] = axis_of(p, i);
    }
    const float one = p.gemma ? 1.0f : 0.0f;
    for (int i = threadIdx.x; i < p.head_dim; i += kRopeWorkers + kRopeLoaders) {
      if (p.q.weight) sh.weight[0][in_planes(i, p.head_dim)] = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(p.q.weight) + i)) + one;
      if (p.k.weight) sh.weight[1][in_planes(i, p.head_dim)] = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(p.k.weight) + i)) + one;
    }
    __syncthreads();
    if (threadIdx.x >= kRopeWorkers)
      load();
    else
      work();
  }
};

template <int DT, int MODE, int LANES>
__global__ void __launch_bounds__(kRopeWorkers + kRopeLoaders, 3) rope_vec(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ typename RopeVec<DT, MODE, LANES>::Shared sh;
  RopeVec<DT, MODE, LANES>{p, plan, sh, raw}.run();
}

template <int DT, int MODE>
const void* vec_of(int dim) {
  switch (dim) {
    case 64: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 4>);
    case 80: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 5>);
    case 96: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 6>);
    case 128: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 8>);
    case 256: return reinterpret_cast<const void*>(&rope_vec<DT, MODE, 16>);
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

RopePlan rope_plan(const RopeParams& p, int sm_count) {
  RopePlan r;
  r.heads = p.q.heads + p.k.heads * (p.k_cache ? 2 : 1);
  const int head = p.head_dim * 2, round = 32 / ((p.head_dim / 8 + 1) / 2) * (kRopeWorkers / 32);  // heads at a time
  // heads of a unit: all, or what fits a stage
  r.split = 1;
  while ((r.heads + r.split - 1) / r.split * head > kRopeRowBytes && r.split < r.heads) r.split *= 2;
  // few tokens: their heads are shared out over the SMs, as long as each unit has a round of them
  while (p.tokens * r.split < sm_count && r.heads > round * r.split) r.split *= 2;
  r.per = (r.heads + r.split - 1) / r.split;
  r.split = (r.heads + r.per - 1) / r.per;
  r.heads_div = fast_div((uint32_t)r.per);
  r.pitch = (p.half + 3) / 4 * 4;
  // Several tokens a unit, as many as make the rounds of a CTA cheapest: a unit has a cost of its own,
  // but the last round should not stand half empty.  (us with units of up to 16, 24, 32 KB: 15412 tokens
  // of 4.6 KB 45, 36, 36; 16384 of 7.7 KB 61, 61, 59; 8324 of 14 KB 54, 54, 51; 2800 of 16 KB, where two
  // tokens make four rounds of three, 23, 23, 26.)
  const int room = kRopeSmem - (!p.pairs && p.half % 8 ? kRopeSkew : 0);
  int64_t best = 0;
  r.step = 1;
  for (int step = 1; step <= (r.split == 1 ? kRopeMaxStep : 1); ++step) {
    const int rows = (step * r.per * head + 127) / 128 * 128, stage = (rows + step * r.pitch * 8 + 127) / 128 * 128;
    if (step > 1 && kStages * stage > room) break;
    const int64_t units = (p.tokens + step - 1) / step, rounds = (units + 3 * sm_count - 1) / (3 * sm_count);
    const int64_t cost = rounds * (step * r.per * head + kRopeUnitCost);
    if (step > 1 && cost >= best) continue;
    best = cost;
    r.step = step;
    r.row_bytes = rows;
    r.stage_bytes = stage;
  }
  r.units = (p.tokens + r.step - 1) / r.step * r.split;
  r.ctas = r.units < (int64_t)3 * sm_count ? (unsigned)r.units : 3u * sm_count;
  return r;
}

size_t rope_smem(const RopePlan& r) { return (size_t)kStages * r.stage_bytes; }

// The largest that rope_plan asks for (one token a unit needs less).
size_t rope_smem_most() { return kRopeSmem; }
static_assert(kStages * (kRopeRowBytes + AR_MAX_HEAD_DIM * 2 + 128 + AR_MAX_HEAD_DIM / 2 * 8 + 128) <= kRopeSmem - kRopeSkew, "one token fits");

}  // namespace ar

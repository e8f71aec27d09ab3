// Append of new keys and values to a paged cache of E4M3 codes: RMSNorm and rotation of k, one scale a
// block and head.
#include "ar_angle.cuh"
#include "ar_append.cuh"
#include "ar_staged.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kScalarThreads = 128;

// Sine and cosine of `pos` times the fraction of a turn, as in the other rotations (ar_angle.cuh), and the eight bits
// that sincospi does not take as a first-order term: off by an ulp or two, so that few codes differ from those of exact angles.
__device__ __forceinline__ void angle_fine(unsigned long long turn, int pos, float* s, float* c) {
  const unsigned long long a = turn * (unsigned long long)(long long)pos;
  const int top = (int)(unsigned)((a + 0x80000000ull) >> 32);  // [-0.5, 0.5) turns in units of 2^-32
  const float head = (float)(top & ~0xff);  // 24 bits
  const float rest = (float)(top & 0xff) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  float s0, c0;
  sincospif(head * 0x1p-31f, &s0, &c0);
  *s = fmaf(c0, rest, s0);
  *c = fmaf(-s0, rest, c0);
}

// 8 bytes that are read once.
__device__ __forceinline__ uint2 ld_v2_once(const void* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Any alignment, stride, head and page size: a warp a token, its values as fp32 in shared memory, computed
// once for the scale and once more for the codes.
template <int DT>
__global__ void __launch_bounds__(kScalarThreads) append_scalar(const __grid_constant__ AppendParams p) {
  constexpr int WARPS = kScalarThreads / 32;
  __shared__ float buf[WARPS][AR_MAX_HEAD_DIM];
  __shared__ float tops[WARPS];
  __shared__ AppendShared sh;
  pdl_wait_and_release();
  append_span<kScalarThreads>(p, 1, sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* x = buf[warp];
  AppendWalk walk;
  walk.start(p, sh, 1);
  AppendUnit u;
  while (walk.next(p, u)) {
    if (u.block < 0) continue;
    for (int task = 0; task < 2 * p.heads; ++task) {
      const bool is_v = task >= p.heads;
      const int h = is_v ? task - p.heads : task;
      const uint16_t* rows = static_cast<const uint16_t*>(is_v ? p.v : p.k) + h * (is_v ? p.v_hs : p.k_hs);
      uint8_t* cache = (is_v ? p.v_cache : p.k_cache) + u.block * (is_v ? p.vc_bs : p.kc_bs) + h * (is_v ? p.vc_hs : p.kc_hs);
      const int64_t ts = is_v ? p.v_ts : p.k_ts, ps = is_v ? p.vc_ps : p.kc_ps;
      const Scales& sc = is_v ? p.v_scale : p.k_scale;
      float* scale = sc.p + u.block * sc.bs + h * sc.hs;
      auto load = [&](int i) {  // the unit's token i, as it is stored, into x
        const uint16_t* src = rows + (u.row + i) * ts;
        float ss = 0.0f;
        __syncwarp();
        for (int e = lane; e < p.head_dim; e += 32) {
          x[e] = to_f32<DT>(ld_u16(src + e));
          ss += x[e] * x[e];
        }
        if (is_v) return;
        if (p.weight) {
          const float rs = rsqrtf(__fdiv_rn(warp_sum(ss), (float)p.head_dim) + p.eps);
          for (int e = lane; e < p.head_dim; e += 32) {
            const float wt = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(p.weight) + e));
            x[e] = x[e] * rs * (p.gemma ? 1.0f + wt : wt);
          }
        }
        __syncwarp();
        for (int f = lane; f < p.half; f += 32) {
          float s, c;
          angle_fine(turn_of(p.inv_freq[f]), p.positions ? p.positions[axis_of(p, f) * p.pos_stride + u.row + i] : u.place + i, &s, &c);
          const int ia = p.pairs ? 2 * f : f, ib = p.pairs ? 2 * f + 1 : f + p.half;
          const float a = x[ia], b = x[ib];
          x[ia] = a * c - b * s;
          x[ib] = b * c + a * s;
        }
        __syncwarp();
      };
      float top = 0.0f;
      for (int i = warp; i < u.n; i += WARPS) {
        load(i);
        for (int e = lane; e < p.head_dim; e += 32) top = fmaxf(top, finite_magnitude(x[e]));
      }
      top = warp_max_magnitude(top);
      const float old = u.held ? clamp_scale(*scale) : kScaleLow;
      __syncthreads();  // every warp has read the scale, and the last task's maxima
      if (lane == 0) tops[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, tops[w]);
      const float now = fmaxf(old, fresh_scale(top)), inv = 1.0f / now;
      if (threadIdx.x == 0) st_f32(scale, now);
      if (u.held && now > old) {
        const float ratio = old * inv;
        for (int i = warp; i < u.held; i += WARPS)
          for (int e = lane; e < p.head_dim; e += 32) {
            uint8_t* at = cache + i * ps + e;
            float a, b;
            from_e4m3x2(*at, a, b);
            st_u8(at, (uint8_t)e4m3x2(a * ratio, 0.0f));
          }
      }
      for (int i = warp; i < u.n; i += WARPS) {
        load(i);
        uint8_t* dst = cache + (u.held + i) * ps;
        for (int e = lane; e < p.head_dim; e += 32) st_u8(dst + e, (uint8_t)e4m3x2(for_code(x[e], inv), 0.0f));
      }
    }
  }
}

constexpr int kVecThreads = 256, kVecWarps = kVecThreads / 32;
constexpr int kSlots = 8;  // rows that a lane holds a part of

// Rows on 8-byte boundaries, heads of a multiple of 8.  A CTA works through units of all (or a share of) the heads of a
// block, so that the angles of its tokens are computed once, into shared memory.  A task is the new keys or the new
// values of one head: `warps` warps take it, LANES lanes a row, each with two chunks of 4 elements: neighbours, or (HALVES)
// chunk c and the one half a rotation on, so that a lane has both elements of each pair.  All rows of a task stay in
// registers from the loads to the codes, with the scale found in between; the next task's rows are on their way
// meanwhile.  Blocks of more tokens than eight warps hold are gone through twice, once for the scale.
//
// The bound should be memory, 6 bytes an element; what it is are instructions (about 24 an element and thread with the
// lanes that heads of 80 leave idle, issue slots 43 % busy) and the waits of 16 warps an SM on each other.  Measured on
// GB300: 16384 tokens x 16 heads of 80, fp16, three axes, 126 MB: 75 us (the general form 1740); 4096 x 8 heads of 128
// in blocks of 64 22 us (blocks of 16: 14.5, of 256, gone through twice: 54); chunks and single
// tokens, 2830 x 8 heads of 128 13 us; 256 single tokens 8 us, 16 5.6 us on the GPU.  Four rows a lane and three or four
// CTAs an SM: 108 and 146 us where eight and two took 99.
template <int DT, int LANES, bool HALVES>
struct AppendVec {
  static constexpr int kRowsAStep = 32 / LANES, kTokens = kSlots * kRowsAStep;  // tokens of a warp

  struct Shared {
    AppendShared span;
    unsigned long long turn[AR_MAX_HEAD_DIM / 2];
    int axis[AR_MAX_HEAD_DIM / 2];
    float weight[AR_MAX_HEAD_DIM];
    float top[kVecWarps];
  };

  const AppendParams& p;
  const AppendPlan& plan;
  Shared& sh;
  float* cosines;  // [tokens][pitch], then the sines
  int lane, warp, sub, task_of_group, row_in_step, c0, c1;
  bool there;
  // of the task whose rows are in `raw`
  int task;
  uint2 raw[kSlots][2];
  float old;

  __device__ __forceinline__ int tokens_a_round() const { return plan.warps * kTokens; }
  __device__ __forceinline__ float* sines() const { return cosines + plan.round_tokens * plan.pitch; }

  __device__ __forceinline__ void angles(const AppendUnit& u, int first) {
    if (!p.half) return;
    const int n = min(u.n - first, tokens_a_round());
    for (int i = threadIdx.x; i < n * p.half; i += kVecThreads) {
      const int t = i / p.half_div, f = i - t * p.half;
      float s, c;
      angle_fine(sh.turn[f], p.positions ? p.positions[sh.axis[f] * p.pos_stride + u.row + first + t] : u.place + first + t, &s, &c);
      cosines[t * plan.pitch + f] = c;
      sines()[t * plan.pitch + f] = s;
    }
  }

  struct Place {  // of a task in a unit
    const uint16_t* rows;
    uint8_t* cache;
    float* scale;
    int64_t ts, ps;
  };
  __device__ __forceinline__ Place place(const AppendUnit& u) const {
    const bool v = task >= p.heads;
    const int h = v ? task - p.heads : task;
    const Scales& sc = v ? p.v_scale : p.k_scale;
    return {static_cast<const uint16_t*>(v ? p.v : p.k) + h * (v ? p.v_hs : p.k_hs),
            (v ? p.v_cache : p.k_cache) + u.block * (v ? p.vc_bs : p.kc_bs) + h * (v ? p.vc_hs : p.kc_hs), sc.p + u.block * sc.bs + h * sc.hs,
            v ? p.v_ts : p.k_ts, v ? p.vc_ps : p.kc_ps};
  }
  __device__ __forceinline__ bool busy() const { return task < 2 * p.heads; }
  __device__ __forceinline__ int token(int first, int slot) const { return first + sub * kTokens + slot * kRowsAStep + row_in_step; }

  // Asks for the rows of a task, from token `first` of the unit on.
  __device__ __forceinline__ void fetch(const AppendUnit& u, int group, int first) {
    task = group * (kVecWarps / plan.warps) + task_of_group;
    if (!busy()) return;
    const Place at = place(u);
    const int t0 = token(first, 0), left = there ? u.n - t0 : 0;
    const uint16_t* src = at.rows + (u.row + t0) * at.ts + c0 * 4;
    const int64_t step = kRowsAStep * at.ts;
    const int other = (c1 - c0) * 4;
#pragma unroll
    for (int k = 0; k < kSlots; ++k, src += step) {
      raw[k][0] = raw[k][1] = make_uint2(0, 0);
      if (k * kRowsAStep < left) {
        raw[k][0] = ld_v2_once(src);
        raw[k][1] = ld_v2_once(src + other);
      }
    }
    old = u.held ? clamp_scale(*reinterpret_cast<const volatile float*>(at.scale)) : kScaleLow;
  }

  // The rows in `raw` as they are stored, two elements a register pair, and the largest magnitude among them.
  __device__ __forceinline__ float values(const AppendUnit& u, int first, uint64_t (&f)[kSlots][4]) {
    const bool v = task >= p.heads;
    const int t0 = token(first, 0), rows = u.n - first - sub * kTokens;  // rows of the warp
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[k][2 * i] = two(to_f32<DT>(raw[k][i].x & 0xffffu), to_f32<DT>(raw[k][i].x >> 16));
        f[k][2 * i + 1] = two(to_f32<DT>(raw[k][i].y & 0xffffu), to_f32<DT>(raw[k][i].y >> 16));
      }
    if (!v && p.weight) {
      uint64_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = two(sh.weight[c0 * 4 + 2 * i], sh.weight[c0 * 4 + 2 * i + 1]);
        w[2 + i] = two(sh.weight[c1 * 4 + 2 * i], sh.weight[c1 * 4 + 2 * i + 1]);
      }
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        if (k * kRowsAStep >= rows) break;
        uint64_t s2 = mul2(f[k][0], f[k][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = fma2(f[k][i], f[k][i], s2);
        float a, b;
        untwo(s2, a, b);
        float ss = a + b;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        // (a division: the reciprocal of a head size that is no power of two would be off by up to 2^-25 in every element of the
        // call, which moved 8 times as many codes as the rest of the arithmetic does)
        const float r = rsqrtf(__fdiv_rn(ss, (float)p.head_dim) + p.eps);
        const uint64_t r2 = two(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[k][i] = mul2(mul2(f[k][i], r2), w[i]);
      }
    }
    if (!v && p.half) {
      // chunk c0's first frequency; pairs of neighbours: two a chunk
      const int f0 = HALVES ? c0 * 4 : c0 * 2;
      if (f0 < p.half && there) {
        const float* at = cosines + (t0 - first) * plan.pitch + f0;
        const int to_sines = plan.round_tokens * plan.pitch;
#pragma unroll
        for (int k = 0; k < kSlots; ++k, at += kRowsAStep * plan.pitch) {
          if (t0 + k * kRowsAStep >= u.n) break;
          if constexpr (HALVES) {  // of a multiple of 4
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(at), s = *reinterpret_cast<const ulonglong2*>(at + to_sines);
            const uint64_t x0 = f[k][0], x1 = f[k][1], y0 = f[k][2], y1 = f[k][3], minus = two(-1.0f, -1.0f);
            f[k][0] = fma2(x0, c.x, mul2(mul2(y0, minus), s.x));
            f[k][1] = fma2(x1, c.y, mul2(mul2(y1, minus), s.y));
            f[k][2] = fma2(y0, c.x, mul2(x0, s.x));
            f[k][3] = fma2(y1, c.y, mul2(x1, s.y));
          } else {
            const float4 c = *reinterpret_cast<const float4*>(at), s = *reinterpret_cast<const float4*>(at + to_sines);
            const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (f0 + i >= p.half) continue;  // an element that does not turn keeps its value, infinities included
              float x, y;
              untwo(f[k][i], x, y);
              f[k][i] = two(x * cs[i] - y * sn[i], y * cs[i] + x * sn[i]);
            }
          }
        }
      }
    }
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        untwo(f[k][i], x, y);
        top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
      }
    if (__any_sync(0xffffffffu, top > 3.402823466e38f)) {  // infinities do not count, and their code is NaN's
      top = 0.0f;
      const float nan = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          untwo(f[k][i], x, y);
          top = fmaxf(top, fmaxf(finite_magnitude(x), finite_magnitude(y)));
          f[k][i] = two(fabsf(x) > 3.402823466e38f ? nan : x, fabsf(y) > 3.402823466e38f ? nan : y);
        }
    }
    return warp_max_magnitude(top);
  }

  // Largest magnitude over a task's warps.
  __device__ __forceinline__ float over_warps(float top) {
    if (plan.warps == 1) return top;
    __syncthreads();
    if (lane == 0) sh.top[warp] = top;
    __syncthreads();
    for (int w = 0; w < plan.warps; ++w) top = fmaxf(top, sh.top[warp - sub + w]);
    return top;
  }

  // Scale, and the codes that the block holds already.
  __device__ __forceinline__ float settle_scale(const AppendUnit& u, const Place& at, float was, float top) {
    const float now = fmaxf(was, fresh_scale(top)), inv = 1.0f / now;
    if (sub == 0 && lane == 0) st_f32(at.scale, now);
    if (u.held && now > was && there) {
      const float ratio = was * inv;
      for (int i = sub * kRowsAStep + row_in_step; i < u.held; i += plan.warps * kRowsAStep) {
        uint8_t* row = at.cache + i * at.ps;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t* q = reinterpret_cast<uint32_t*>(row + (k ? c1 : c0) * 4);
          float a, b, c, d;
          from_e4m3x2(*q & 0xffffu, a, b);
          from_e4m3x2(*q >> 16, c, d);
          *q = e4m3x2(a * ratio, b * ratio) | (e4m3x2(c * ratio, d * ratio) << 16);
        }
      }
    }
    return inv;
  }

  __device__ __forceinline__ void store(const AppendUnit& u, const Place& at, int first, const uint64_t (&f)[kSlots][4], float inv) {
    const int t0 = token(first, 0), left = there ? u.n - t0 : 0, other = (c1 - c0) * 4;
    uint8_t* dst = at.cache + (u.held + t0) * at.ps + c0 * 4;
    const int64_t step = kRowsAStep * at.ps;
    const uint64_t inv2 = two(inv, inv);
#pragma unroll
    for (int k = 0; k < kSlots; ++k, dst += step) {
      if (k * kRowsAStep >= left) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float a, b, c, d;
        untwo(mul2(f[k][2 * i], inv2), a, b);
        untwo(mul2(f[k][2 * i + 1], inv2), c, d);
        *reinterpret_cast<uint32_t*>(dst + (i ? other : 0)) = e4m3x2(a, b) | (e4m3x2(c, d) << 16);
      }
    }
  }

  __device__ __forceinline__ void run() {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    sub = warp % plan.warps;
    task_of_group = warp / plan.warps;
    row_in_step = lane / LANES;
    const int c = lane % LANES, hb = p.half / 4;
    there = c * 8 < p.head_dim;
    const bool turns = HALVES && c < hb;
    c0 = turns ? c : 2 * c;
    c1 = turns ? c + hb : 2 * c + 1;
    if (!there) c0 = c1 = 0;
    const int a_group = kVecWarps / plan.warps, groups = (2 * p.heads + a_group - 1) / a_group;
    AppendWalk walk;
    walk.start(p, sh.span, plan.parts);
    AppendUnit u;
    uint64_t f[kSlots][4];
    while (walk.next(p, u)) {
      if (u.block < 0) continue;
      const int g0 = u.part * groups / plan.parts, g1 = (u.part + 1) * groups / plan.parts;
      const bool keys = g0 * a_group < p.heads;  // the share has keys
      if (u.n <= tokens_a_round()) {
        fetch(u, g0, 0);
        __syncthreads();  // the unit before is done with the angles
        if (keys) angles(u, 0);
        __syncthreads();
        for (int g = g0; g < g1; ++g) {
          const bool mine = busy();
          const Place at = place(u);
          const float was = old;
          float top = mine ? values(u, 0, f) : 0.0f;
          if (g + 1 < g1) fetch(u, g + 1, 0);
          top = over_warps(top);
          if (mine) store(u, at, 0, f, settle_scale(u, at, was, top));
        }
      } else {
        for (int g = g0; g < g1; ++g) {
          const bool turn = g * a_group < p.heads;
          float top = 0.0f, inv = 0.0f;
          for (int pass = 0; pass < 2; ++pass) {
            for (int first = 0; first < u.n; first += tokens_a_round()) {
              __syncthreads();
              if (turn) angles(u, first);
              fetch(u, g, first);
              __syncthreads();
              const float part = busy() ? values(u, first, f) : 0.0f;
              if (pass == 0)
                top = fmaxf(top, part);
              else if (busy())
                store(u, place(u), first, f, inv);
            }
            if (pass == 0) {
              const float was = old;
              top = over_warps(top);
              __syncthreads();  // every warp has read the scale
              if (busy()) inv = settle_scale(u, place(u), was, top);
            }
          }
        }
      }
    }
  }
};

template <int DT, int LANES, bool HALVES>
__global__ void __launch_bounds__(kVecThreads, 2) append_vec(const __grid_constant__ AppendParams p, const __grid_constant__ AppendPlan plan) {
  using V = AppendVec<DT, LANES, HALVES>;
  extern __shared__ __align__(16) float angles[];
  __shared__ typename V::Shared sh;
  pdl_wait_and_release();
  for (int i = threadIdx.x; i < p.half; i += kVecThreads) {
    sh.turn[i] = turn_of(p.inv_freq[i]);
    sh.axis[i] = axis_of(p, i);
  }
  if (p.weight)
    for (int i = threadIdx.x; i < p.head_dim; i += kVecThreads) {
      const float w = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(p.weight) + i));
      sh.weight[i] = p.gemma ? 1.0f + w : w;
    }
  append_span<kVecThreads>(p, plan.parts, sh.span);
  V{p, plan, sh, angles}.run();
}

int lanes_of(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

}  // namespace

AppendPlan append_plan(const AppendParams& p, int sm_count) {
  AppendPlan plan;
  const int tokens = kSlots * 32 / lanes_of(p.head_dim), page = (int)p.page.d;
  plan.warps = 1;
  while (plan.warps < kVecWarps && plan.warps * tokens < page) plan.warps *= 2;
  plan.round_tokens = plan.warps * tokens < page ? plan.warps * tokens : page;
  plan.pitch = (p.half + 3) / 4 * 4;
  // blocks that can get tokens: a request's first and last one, and whole ones between
  const int64_t most = p.tokens / page + 2 * (int64_t)p.requests < p.tokens ? p.tokens / page + 2 * (int64_t)p.requests : p.tokens;
  // shares of a block's heads, until there are about six units a resident CTA (16384 video tokens with two 107 us)
  const int groups = (2 * p.heads + kVecWarps / plan.warps - 1) / (kVecWarps / plan.warps);
  const int64_t usual = p.tokens / page + p.requests < p.tokens ? p.tokens / page + p.requests : p.tokens;
  plan.parts = 1;
  while (plan.parts < groups && usual * plan.parts < 12 * sm_count) ++plan.parts;
  const int64_t grid = most * plan.parts;
  plan.ctas = (unsigned)(grid < (int64_t)sm_count * 2 ? grid : (int64_t)sm_count * 2);
  return plan;
}

size_t append_smem(const AppendPlan& plan) { return (size_t)plan.round_tokens * plan.pitch * 8; }
size_t append_smem_most() { return 64 * 1024; }

namespace {

template <int DT, bool HALVES>
const void* vec_of(int lanes) {
  return lanes == 8    ? reinterpret_cast<const void*>(&append_vec<DT, 8, HALVES>)
         : lanes == 16 ? reinterpret_cast<const void*>(&append_vec<DT, 16, HALVES>)
                       : reinterpret_cast<const void*>(&append_vec<DT, 32, HALVES>);
}

}  // namespace

const void* append_vec_kernel(bool bf16, int head_dim, bool halves) {
  const int lanes = lanes_of(head_dim);
  if (halves) return bf16 ? vec_of<kBF16, true>(lanes) : vec_of<kF16, true>(lanes);
  return bf16 ? vec_of<kBF16, false>(lanes) : vec_of<kF16, false>(lanes);
}

const void* append_scalar_kernel(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&append_scalar<kBF16>) : reinterpret_cast<const void*>(&append_scalar<kF16>);
}

}  // namespace ar

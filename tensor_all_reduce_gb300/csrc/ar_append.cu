// Append of new keys and values to a paged cache of E4M3 codes: RMSNorm and rotation of k, one scale a
// block and head.
#include "ar_angle.cuh"
#include "ar_append.cuh"
#include "ar_staged.cuh"

namespace ar {
namespace {

constexpr int kScalarThreads = 128;

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
          const float rs = rsqrtf(warp_sum(ss) * p.inv_dim + p.eps);
          for (int e = lane; e < p.head_dim; e += 32) {
            const float wt = to_f32<DT>(ld_u16(static_cast<const uint16_t*>(p.weight) + e));
            x[e] = x[e] * rs * (p.gemma ? 1.0f + wt : wt);
          }
        }
        __syncwarp();
        for (int f = lane; f < p.half; f += 32) {
          float s, c;
          angle(turn_of(p.inv_freq[f]), p.positions ? p.positions[axis_of(p, f) * p.pos_stride + u.row + i] : u.place + i, &s, &c);
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

}  // namespace

const void* append_scalar_kernel(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&append_scalar<kBF16>) : reinterpret_cast<const void*>(&append_scalar<kF16>);
}

}  // namespace ar

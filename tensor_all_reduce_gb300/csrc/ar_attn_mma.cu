// Paged attention, general form: any head size up to 256, page size, stride and alignment.
//
// One CTA of four warps takes 64 query rows (16 a warp) against tiles of 64 keys: scores and
// the weighted sum by 16 x 8 x 16 matrix instructions on tiles in shared memory, the softmax's
// running maximum and sum in registers, each key and value read once an item.  Keys are gathered
// row by row through the block table, so pages may end anywhere in a tile.
//
// It serves what the tensor-core kernel's copies cannot take (odd head sizes, strides, page sizes) and
// is bound by the issue of its matrix instructions and of the gathers, nothing in it being
// asynchronous.  With aligned rows and pages of 12 (of 1) tokens: 4096 tokens over 28000 (12 heads, 2 key
// heads of 128) 6.0 (6.2) ms against 0.51 ms in pages of 64, 64 single tokens over up to 9000 keys (48
// heads, 8 key heads) 1.05 (1.11) ms against 0.22 ms in pages of 16; element by element 8.8 and 1.26 ms.
// Over 8-bit caches 9.0 and 1.36 ms in pages of 12, element by element 10.8 and 1.6 ms.
#include <type_traits>

#include "ar_attn.cuh"
#include "ar_e4m3.cuh"

namespace ar {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 128;
constexpr int kJoinThreads = 256;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == kBF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One row of head_dim elements into shared memory, the rest of the padded row zero; src NULL: zeros.
template <int DP>
__device__ __forceinline__ void fill_row(const AttnParams& p, uint16_t* dst, const uint16_t* src, int part, int parts) {
  for (int c = part; c < DP / 8; c += parts) {
    uint4 v = make_uint4(0, 0, 0, 0);
    const int e = c * 8;
    if (src && e < p.head_dim) {
      if (p.vec) {
        v = ld_keep(src + e);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = e + i < p.head_dim ? ld_u16(src + e + i) : 0;
        v = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
      }
    }
    *reinterpret_cast<uint4*>(dst + e) = v;
  }
}

// The same for a row of E4M3 codes, whose values both 16-bit types hold.
template <int DT, int DP>
__device__ __forceinline__ void fill_codes(const AttnParams& p, uint16_t* dst, const uint8_t* src, int part, int parts) {
  for (int c = part; c < DP / 8; c += parts) {
    const int e = c * 8;
    uint32_t w[4] = {0, 0, 0, 0};
    if (src && e < p.head_dim) {
      uint32_t codes[2] = {0, 0};
      if (p.vec) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + e);
        codes[0] = v.x;
        codes[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < p.head_dim) codes[i >> 2] |= (uint32_t)src[e + i] << (8 * (i & 3));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        from_e4m3x2(codes[i >> 1] >> (16 * (i & 1)), a, b);
        w[i] = pack2<DT>(a, b);
      }
    }
    *reinterpret_cast<uint4*>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// FP8: the cache holds E4M3 codes.  The codes are the products' operands, both 16-bit types hold them.  A
// key's score takes its block's k scale; its v scale joins the weight, which is held relative to the largest
// product of the two in the row, so that scales of any size neither overflow nor drown: with t = log2(vs),
//   w_j = 2^(s_j + t_j - m),  o = sum w_j c_j,  l = sum w_j / vs_j,  out = o / l.
// In fp16, whose steps end at 2^-24, m is 14 below the largest: a weight is then off by 2^-39 of that at most (with the largest at 1,
// very many equal weights that are 2^-24 of it kept 1 to 7 % too little or too much of their sum).
template <int DT, int DP, bool FP8>
__global__ void __launch_bounds__(kThreads) attn_mma(const __grid_constant__ AttnParams p) {
  constexpr int LD = DP + 8;  // 16 bytes of padding: the eight rows of a matrix load fall into different banks
  extern __shared__ __align__(16) uint16_t smem[];
  uint16_t* sq = smem;
  uint16_t* sk = sq + kRows * LD;
  uint16_t* sv = sk + kKeys * LD;
  __shared__ SpanShared span;
  constexpr float kLift = FP8 && DT == kF16 ? 14.0f : 0.0f;
  __shared__ float4 scales[FP8 ? kKeys : 1];  // of a key: k scale, log2 and reciprocal of the v scale
  pdl_wait_and_release();
  find_span<kRows, kKeys, kThreads>(p, span);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool goes_on = false;
  Walk<kRows, kKeys> walk;
  walk.start(span);
  Item it;
  while (walk.next(p, it)) {
    __syncthreads();
    for (int r = threadIdx.x >> 2; r < kRows; r += kThreads / 4) {
      const int row = it.qt * kRows + r;
      const uint16_t* src = nullptr;
      if (row < it.rows) {
        const int t = row / p.group, g = row - t * (int)p.group.d;
        src = static_cast<const uint16_t*>(p.q) + (int64_t)(it.q.q0 + t) * p.q_ts + (int64_t)(it.h * (int)p.group.d + g) * p.q_hs;
      }
      fill_row<DP>(p, sq + r * LD, src, threadIdx.x & 3, 4);
    }
    // the two rows of this lane
    RowView view[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) view[i] = row_view(p, it, it.qt * kRows + warp * 16 + (lane >> 2) + i * 8);
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const KeyRange keys = tile_keys<kRows>(p, it.q, it.qt);

    for (int ti = it.begin; ti < it.end; ++ti) {
      const int key0 = it.range.tile(ti) * kKeys;
      __syncthreads();
      for (int r = threadIdx.x >> 2; r < kKeys; r += kThreads / 4) {
        const int key = key0 + r;
        using Elem = std::conditional_t<FP8, uint8_t, uint16_t>;
        const Elem *k = nullptr, *v = nullptr;
        float4 scale = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        if (keys.sees(it.q, key)) {  // the others are zeros: a weight of 0 does not cancel a NaN
          int off;
          const int64_t b = block_of(p, it, key, off);
          if (b >= 0) {
            k = static_cast<const Elem*>(p.k) + b * p.k_bs + off * p.k_ps + it.h * p.k_hs;
            v = static_cast<const Elem*>(p.v) + b * p.v_bs + off * p.v_ps + it.h * p.v_hs;
            if constexpr (FP8) scale = load_scales(p, b, it.h);
          }
        }
        if constexpr (FP8) {
          if ((threadIdx.x & 3) == 0) scales[r] = scale;
          fill_codes<DT, DP>(p, sk + r * LD, k, threadIdx.x & 3, 4);
          fill_codes<DT, DP>(p, sv + r * LD, v, threadIdx.x & 3, 4);
        } else {
          fill_row<DP>(p, sk + r * LD, k, threadIdx.x & 3, 4);
          fill_row<DP>(p, sv + r * LD, v, threadIdx.x & 3, 4);
        }
      }
      __syncthreads();

      float s[kKeys / 8][4];
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t a[4];
        ldsm4(a, smem_u32(sq + (warp * 16 + (lane & 15)) * LD + kk * 16 + (lane >> 4) * 8));
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j) {
          uint32_t b[4];
          ldsm4(b, smem_u32(sk + (j * 16 + (lane >> 4) * 8 + (lane & 7)) * LD + kk * 16 + ((lane >> 3) & 1) * 8));
          mma<DT>(s[2 * j], a, b[0], b[1]);
          mma<DT>(s[2 * j + 1], a, b[2], b[3]);
        }
      }
      // scores in log2 units; what a row does not see is -inf whatever the product gave
      float top[2] = {m[0] + kLift, m[1] + kLift};
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + j * 8 + (lane & 3) * 2 + (e & 1);
          const RowView& w = view[e >> 1];
          if constexpr (FP8) {
            const float4 c = scales[j * 8 + (lane & 3) * 2 + (e & 1)];
            s[j][e] = visible(it, w, key) ? bend(p, w, s[j][e] * c.x, key) + c.y : -INFINITY;
          } else {
            s[j][e] = visible(it, w, key) ? bend(p, w, s[j][e], key) : -INFINITY;
          }
          top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
        }
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        top[i] -= kLift;
        base[i] = top[i] == -INFINITY ? 0.0f : top[i];
        const float shrink = ex2(m[i] - base[i]);  // m = -inf: 0
        m[i] = top[i];
        l[i] *= shrink;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          o[j][2 * i] *= shrink;
          o[j][2 * i + 1] *= shrink;
        }
      }
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j][e] = ex2(s[j][e] - base[e >> 1]);
          if constexpr (FP8)
            l[e >> 1] = fmaf(s[j][e], scales[j * 8 + (lane & 3) * 2 + (e & 1)].z, l[e >> 1]);
          else
            l[e >> 1] += s[j][e];
        }
      // weights rounded to the 16-bit type for the second product; their sum l is of the unrounded ones
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk) {
        const uint32_t a[4] = {pack2<DT>(s[2 * kk][0], s[2 * kk][1]), pack2<DT>(s[2 * kk][2], s[2 * kk][3]),
                               pack2<DT>(s[2 * kk + 1][0], s[2 * kk + 1][1]), pack2<DT>(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          uint32_t b[4];
          ldsm4t(b, smem_u32(sv + (kk * 16 + (lane & 15)) * LD + j * 16 + (lane >> 4) * 8));
          mma<DT>(o[2 * j], a, b[0], b[1]);
          mma<DT>(o[2 * j + 1], a, b[2], b[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int local = warp * 16 + (lane >> 2) + i * 8, row = it.qt * kRows + local;
      if (row >= it.rows) continue;
      if (whole) {
        const int t = row / p.group, head = it.h * (int)p.group.d + row - t * (int)p.group.d;
        const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
        uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          const int e = j * 8 + (lane & 3) * 2;
          if (p.vec) {
            if (e < p.head_dim) *reinterpret_cast<uint32_t*>(dst + e) = pack2<DT>(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
          } else {
            if (e < p.head_dim) st_u16(dst + e, round1<DT>(o[j][2 * i] * inv));
            if (e + 1 < p.head_dim) st_u16(dst + e + 1, round1<DT>(o[j][2 * i + 1] * inv));
          }
        }
        if (p.lse && (lane & 3) == 0)
          p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * kRows + local;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          const int e = j * 8 + (lane & 3) * 2;
          if (e < p.part_dim) *reinterpret_cast<float2*>(p.part_o + at * p.part_dim + e) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
        }
        if ((lane & 3) == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m[i], l[i]);
      }
    }
    if (it.first && !it.last) {
      goes_on = true;
      if (threadIdx.x == 0) write_header(p, span, &it);
    }
  }
  if (threadIdx.x == 0 && !goes_on) write_header(p, span, nullptr);
}

// A partial softmax: sum and weight sum relative to the maximum m (log2 units).
struct Part {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void join(Part& a, float m, float l, const float4& o) {
  const float top = fmaxf(a.m, m), base = top == -INFINITY ? 0.0f : top;
  const float x = ex2(a.m - base), y = ex2(m - base);
  a.m = top;
  a.l = a.l * x + l * y;
  a.o = make_float4(a.o.x * x + o.x * y, a.o.y * x + o.y * y, a.o.z * x + o.z * y, a.o.w * x + o.w * y);
}

// Joins the parts of the items that more than one span holds: the blocks (c, ...) serve the item
// that begins in span c and goes on; its parts are slot 1 of span c and slot 0 of the spans behind
// it.  Many rows with few parts (chunks): a warp takes whole rows.  Few rows with many parts
// (single tokens): a block takes a row, its warps share the parts.
template <int DT>
__global__ void __launch_bounds__(kJoinThreads) attn_combine(const __grid_constant__ AttnParams p) {
  constexpr int WARPS = kJoinThreads / 32, AHEAD = 8;
  __shared__ Part sh[WARPS][32];
  pdl_wait_and_release();
  const int c = blockIdx.x;
  const int* h = p.headers + (int64_t)c * kHeaderInts;
  const int end = h[0];
  if (end == 0) return;
  const int q0 = h[1], rows = h[2], row_base = h[3] * p.tile_rows, head0 = h[4] * (int)p.group.d;
  const int local_rows = min(rows - row_base, p.tile_rows), parts = end - c + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // rounds of loads one after another in either way
  const int by_rows = (local_rows + WARPS * (int)gridDim.y - 1) / (WARPS * (int)gridDim.y) * ((parts + AHEAD - 1) / AHEAD);
  const int by_parts = (local_rows + (int)gridDim.y - 1) / (int)gridDim.y * ((parts + WARPS * AHEAD - 1) / (WARPS * AHEAD));
  const bool share = by_parts < by_rows;  // the warps share a row's parts
  const int step = share ? gridDim.y : gridDim.y * WARPS;
  for (int local = share ? blockIdx.y : blockIdx.y * WARPS + warp; local < local_rows; local += step) {
    const int row = row_base + local;
    const int t = row / p.group, head = head0 + row - t * (int)p.group.d;
    uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)(q0 + t) * p.o_ts + (int64_t)head * p.o_hs;
    for (int e0 = 0; e0 < p.part_dim; e0 += 128) {
      const int e = e0 + lane * 4;
      Part a = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      const int stride = share ? WARPS : 1;
      for (int i0 = c + (share ? warp : 0); i0 <= end; i0 += stride * AHEAD) {
        float2 ml[AHEAD];
        float4 o[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const int i = i0 + k * stride;
          ml[k] = make_float2(-INFINITY, 0.0f);
          o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (i <= end) {
            const int64_t at = ((int64_t)i * 2 + (i == c ? 1 : 0)) * p.tile_rows + local;
            ml[k] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
            if (e < p.part_dim) o[k] = *reinterpret_cast<const float4*>(p.part_o + at * p.part_dim + e);
          }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) join(a, ml[k].x, ml[k].y, o[k]);
      }
      if (share) {
        __syncthreads();
        sh[warp][lane] = a;
        __syncthreads();
        if (warp != 0) continue;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) join(a, sh[w][lane].m, sh[w][lane].l, sh[w][lane].o);
      }
      const float inv = a.l == 0.0f ? 0.0f : 1.0f / a.l;
      const float f[4] = {a.o.x * inv, a.o.y * inv, a.o.z * inv, a.o.w * inv};
      if (p.vec) {
        if (e < p.head_dim) st_v2(dst + e, make_uint2(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < p.head_dim) st_u16(dst + e + j, round1<DT>(f[j]));
      }
      if (p.lse && e == 0)
        p.lse[(int64_t)(q0 + t) * p.q_heads + head] = a.l == 0.0f ? -INFINITY : (a.m + log2f(a.l)) * 0.69314718055994531f;
    }
  }
}

template <int DT, bool FP8>
const void* mma_of(int dp) {
  switch (dp) {
    case 64: return reinterpret_cast<const void*>(&attn_mma<DT, 64, FP8>);
    case 128: return reinterpret_cast<const void*>(&attn_mma<DT, 128, FP8>);
    case 256: return reinterpret_cast<const void*>(&attn_mma<DT, 256, FP8>);
  }
  return nullptr;
}

}  // namespace

const void* attn_mma_kernel(bool bf16, int padded_dim, bool fp8) {
  if (fp8) return bf16 ? mma_of<kBF16, true>(padded_dim) : mma_of<kF16, true>(padded_dim);
  return bf16 ? mma_of<kBF16, false>(padded_dim) : mma_of<kF16, false>(padded_dim);
}

const void* attn_combine_kernel(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&attn_combine<kBF16>) : reinterpret_cast<const void*>(&attn_combine<kF16>);
}

}  // namespace ar

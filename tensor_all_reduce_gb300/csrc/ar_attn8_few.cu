// Paged attention over a cache of E4M3 codes for few rows a request (single tokens, drafts): the products turned
// around, so that keys and values, not queries, are the 128-row operand.
//
// An item is up to 16 query rows of one request and key head.  With X = hi + mid / 16 + lo / 256 in three E4M3
// parts (14 bits), side by side as 48 columns, a tile of 128 keys is two products of 8-bit matrix instructions:
//   scores   S[key, (part, row)] = K[key, d] Q[(part, row), d]          128 x 48 x head
//   sums     O[d, (part, row)]  += V[key, d]^T W[(part, row), key]      128 x 48 x 128, for each 128 of the head
// Each byte of keys and values is thus read from shared memory once, as it came, and the tensor core's time and
// the softmax's do not count 128 rows where there are six.  The kernel that keeps queries as the 128-row operand
// reads keys twice (two parts), turns values to fp16 and was bound by that traffic in shared memory: 64 single
// tokens over up to 9000 keys, 48 heads, 8 key heads of 128: 273 us.
//
// A thread of the softmax warpgroup owns a key: it adds up the parts of the key's scores, and its weights, times
// the v scale as in ar_attn8_tma.cu, go to shared memory as parts.  The references m of the 16 rows are the same
// in all threads; they move only when some weight of a tile would exceed 2^8 (one vote a tile), and then so that
// the largest becomes 2^6, which keeps weights down to 2^-24 of the largest.
//
// Two CTAs an SM, 256 threads each: a warpgroup for the softmax; warps for the matrix instructions, keys, values
// and scales.  Work division, parts of split items and their joining are the other kernels'.  Every wait is bounded.
#include <cuda.h>

#include "ar_attn8.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kRows = kAttn8FewRows, kParts = 3, kColumns = kParts * kRows;
constexpr int kThreads = 256;
constexpr int kMmaWarp = 4, kLoadWarp = 5;  // kLoadWarp + 1: values; the last: scales
constexpr uint32_t kTmemCols = 256;                         // two score buffers and two sums, 64 columns each
constexpr int kOperandBytes = kColumns * 128;               // queries (of 128 elements) or weights: rows of 128 bytes
constexpr float kPart = 16.0f, kPartInv = 0.0625f;          // a part holds the rest of the one before, times 16

template <int DP>
struct Few {
  static constexpr int kRows = ar::kAttn8FewRows;
  static constexpr int kUnits = DP / 128;
  static constexpr int kKeySlots = 3, kValueSlots = 2;  // two CTAs' fill an SM's shared memory
  static constexpr int kBytes = (kUnits + 2) * kOperandBytes + (kKeySlots + kValueSlots) * kUnitBytes;
};

struct Bars {
  Ring k, v;
  uint64_t q;          // queries stored
  uint64_t s[2];       // scores ready
  uint64_t p[2];       // weights stored
  uint64_t o[2];       // sum complete, of a tile
  uint64_t sc_full[kScaleTiles], sc_empty[kScaleTiles];
  uint64_t drain;
  uint32_t tmem;
  int stop;
};

struct FewShared {
  SpanShared span;
  Bars b;
  float4 scales[kScaleTiles][kScaleGroups];
  float factor[kRows];           // of a row: what q was divided by
  int see_lo[kRows], see_hi[kRows], pos[kRows];
  float slope[kRows];
  float top[4][kRows];           // of a warp
};

// The three parts of four floats.
__device__ __forceinline__ void parts4(float a, float b, float c, float d, uint32_t (&part)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    part[i] = codes4<false>(a, b, c, d);
    if (i + 1 == kParts) break;
    minus_codes4(part[i], a, b, c, d);
    a *= kPart, b *= kPart, c *= kPart, d *= kPart;
  }
}

__device__ __forceinline__ uint32_t few_desc(bool a_rows_along_k) {
  return (1u << 4) | ((a_rows_along_k ? 1u : 0u) << 15) | ((uint32_t)(kColumns >> 3) << 17) | ((128u >> 4) << 24);
}

template <int DP>
__device__ void few_mma_role(const AttnParams& p, FewShared& sh, uint32_t queries, uint32_t weights, uint32_t keys, uint32_t values, uint32_t tmem) {
  using S = Few<DP>;
  Bars& b = sh.b;
  const int lane = threadIdx.x & 31;
  const int ksteps = (p.head_dim + 31) / 32;
  const uint32_t idesc_s = few_desc(false), idesc_o = few_desc(true);
  const uint64_t q_desc = matrix_desc(queries, 16), w_desc = matrix_desc(weights, 16), k_desc = matrix_desc(keys, 16), v_desc = matrix_desc(values, kUnitBytes);
  const bool one = elect_one();
  Walk<S::kRows, kKeys> walk;
  walk.start(sh.span);
  Item it = {};
  uint32_t ks = 0, kr = 0, vs = 0, vr = 0;  // slots and rounds in turn
  uint32_t items = 0, g = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  auto scores = [&](uint32_t x) {
    for (int u = 0; u < S::kUnits; ++u) {
      if (!wait(&b.k.full[ks], kr & 1)) return;
      if (one) {
        const uint64_t a = k_desc + ks * (kUnitBytes / 16), q = q_desc + u * (kOperandBytes / 16);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (u * 4 + s < ksteps) mma_8bit(tmem + x * 64, a + s * 2, q + s * 2, idesc_s, u > 0 || s > 0);
        mma_commit(&b.k.empty[ks]);
      }
      if (++ks == S::kKeySlots) ks = 0, ++kr;
    }
    if (one) mma_commit(&b.s[x]);
  };
  // Values behind the request's end become zeros: the rest of a box holds whatever the cache does, and a weight
  // of 0 does not cancel a NaN.
  auto clear_tail = [&](int left) {
    if (left >= kKeys) return;
    const int lo = max(left, 0), hi = min((lo + p.box_rows - 1) / p.box_rows * p.box_rows, kKeys);
    const uint32_t v = values + vs * kUnitBytes;
    for (int x = lo * 8 + lane; x < hi * 8; x += 32) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + x * 16), "r"(0) : "memory");
    fence_proxy_async_smem();
    __syncwarp();
  };
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    if (!wait(&b.q, items & 1)) break;
    scores(g & 1);
    for (int i = 0; ok && i < nt; ++i) {
      if (i + 1 < nt) scores((g + i + 1) & 1);
      if (!ok) break;
      const uint32_t x = (g + i) & 1;
      if (!wait(&b.p[x], ((g + i) >> 1) & 1)) break;
      for (int u = 0; u < S::kUnits; ++u) {
        if (!wait(&b.v.full[vs], vr & 1)) break;
        clear_tail(it.q.len - it.range.tile(it.begin + i) * kKeys);
        if (one) {
          const uint64_t a = v_desc + vs * (kUnitBytes / 16), w = w_desc + x * (kOperandBytes / 16);
          if (u * 128 < p.head_dim)
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_8bit(tmem + 128 + u * 64, a + ((s * 32 * 128) >> 4), w + s * 2, idesc_o, i > 0 || s > 0);
          mma_commit(&b.v.empty[vs]);
        }
        if (++vs == S::kValueSlots) vs = 0, ++vr;
      }
      if (!ok) break;
      if (one) mma_commit(&b.o[x]);
    }
    g += nt;
    ++items;
  }
  if (!ok) {  // matrix instructions in flight end before tensor memory is freed
    if (one) mma_commit(&b.drain);
    mbar_wait_bounded(&b.drain, 0, p.wait_cycles);
  }
}

// 48 columns of tensor memory: the parts of 16 rows, added up.
__device__ __forceinline__ void load_rows(uint32_t addr, float (&f)[kRows]) {
  uint32_t a[32], c[16];
  tmem_ld32(a, addr);
  tmem_ld16(c, addr + 32);
  tmem_wait_ld();
  settle(a);
  settle16(c);
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    f[r] = fmaf(fmaf(__uint_as_float(c[r]), kPartInv, __uint_as_float(a[kRows + r])), kPartInv, __uint_as_float(a[r]));
}

template <int DT, int DP>
__device__ void few_softmax_role(const AttnParams& p, FewShared& sh, uint32_t queries, uint32_t weights, uint32_t tmem) {
  using S = Few<DP>;
  Bars& b = sh.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
  const bool bent = p.cap_log2 > 0.0f || p.slopes || !(p.scale_log2 > 0.0f);
  Walk<S::kRows, kKeys> walk;
  walk.start(sh.span);
  uint32_t g = 0;
  bool ok = true, goes_on = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  auto together = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
  auto any = [](bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbar.red.or.pred b, 2, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}" : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
  };
  // Queries, 16 bytes a lane; the rows of the next item are asked for before the last sums of this one are read.
  constexpr int kRowLanes = DP / 8, kStep = 32 / kRowLanes, kRounds = kRows / 4 / kStep;
  const int col = (lane % kRowLanes) * 8, sub = lane / kRowLanes;
  uint4 raw[kRounds];
  auto fetch = [&](const Item& it) {
    const int base = it.qt * S::kRows, rows = it.rows - base;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)it.q.q0 * p.q_ts + (int64_t)it.h * (int)p.group.d * p.q_hs;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int r = warp * (kRows / 4) + k * kStep + sub;
      raw[k] = make_uint4(0, 0, 0, 0);
      if (r < rows && col < p.head_dim) {
        const int t = (base + r) / p.group, e = base + r - t * (int)p.group.d;
        raw[k] = ld_keep(q + t * p.q_ts + e * p.q_hs + col);
      }
    }
  };
  // Rows that the item does not have are zeros.
  auto queries_loaded = [&](const Item& it) {
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int r = warp * (kRows / 4) + k * kStep + sub;
      float f[8];
      unpack8<DT>(raw[k], f);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_magnitude(f[i]));
#pragma unroll
      for (int o = kRowLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^(e - 127): the power of two that brings the largest element to 224 .. 448
      const int e = max((int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8, 1);
      const float inv = __uint_as_float((unsigned)(254 - e) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = for_code(f[i], inv);
      uint32_t lo[kParts], hi[kParts];
      parts4(f[0], f[1], f[2], f[3], lo);
      parts4(f[4], f[5], f[6], f[7], hi);
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        const int n = x * kRows + r;
        sts_v2(queries + (col >> 7) * kOperandBytes + n * 128 + ((((col & 127) >> 4) ^ (n & 7)) << 4) + (col & 8), lo[x], hi[x]);
      }
      if (col == 0) {
        const RowView v = row_view(p, it, it.qt * S::kRows + r);
        const float factor = __uint_as_float((unsigned)e << 23);
        // within these bounds products of 0 stay 0, and what a k scale can add stays finite
        sh.factor[r] = bent ? factor : fminf(fmaxf(factor * p.scale_log2, 0x1p-90f), 0x1p95f);
        sh.pos[r] = v.pos;
        sh.slope[r] = v.slope;
        const bool there = it.qt * S::kRows + r < it.rows;  // else: sees all, so that a tile need not be masked for it
        sh.see_lo[r] = there ? v.see_lo : 0;
        sh.see_hi[r] = there ? v.see_hi : 0x7fffffff;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.q);
    together();  // what the rows see is there for all
  };
  Item it = {}, later = {};
  bool have = walk.next(p, it);
  if (have) {
    fetch(it);
    queries_loaded(it);
  }
  while (have) {
    const int nt = it.end - it.begin, row0 = it.qt * S::kRows, rows = min(it.rows - row0, S::kRows);
    float m[kRows], l[kRows], factor[kRows];
    int lo = 0, hi = 0x7fffffff;  // keys that all rows see
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
      factor[r] = sh.factor[r];
      lo = max(lo, sh.see_lo[r]);
      hi = min(hi, sh.see_hi[r]);
    }
    for (int i = 0; i < nt; ++i) {
      const uint32_t c = g + i, x = c & 1, phase = (c >> 1) & 1, stage = c % kScaleTiles;
      // (The four warps meet at barriers that do not run out, so they leave together: a wait that ran out is part of
      // the next vote.)
      wait(&b.s[x], phase);
      wait(&b.sc_full[stage], (c / kScaleTiles) & 1);
      const float4 e = sh.scales[stage][tid >> 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.sc_empty[stage]);
      float s[kRows];
      load_rows(lanes + x * 64, s);
      const int key0 = it.range.tile(it.begin + i) * kKeys, key = key0 + tid, prefix = it.q.prefix;
      const bool edge = !((key0 + kKeys <= hi && key0 >= lo) || key0 + kKeys <= prefix);
      if (bent) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          RowView v;
          v.pos = sh.pos[r];
          v.slope = sh.slope[r];
          s[r] = bend(p, v, s[r] * (factor[r] * e.x), key) + e.y;
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r] = fmaf(s[r], factor[r] * e.x, e.y);
      }
      if (edge)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (!(key < prefix || (key < sh.see_hi[r] && key >= sh.see_lo[r]))) s[r] = -INFINITY;
      bool grown = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) grown = grown || s[r] > m[r] + 8.0f;  // m = -inf: any finite score
      if (any(grown || !ok)) {
        if (any(!ok)) {
          ok = false;
          break;
        }
        float shrink[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float top = s[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (lane == r) sh.top[warp][r] = top;
        }
        together();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float high = fmaxf(fmaxf(sh.top[0][r], sh.top[1][r]), fmaxf(sh.top[2][r], sh.top[3][r]));
          const bool moves = high > m[r] + 8.0f;
          shrink[r] = moves ? ex2(m[r] - (high - 6.0f)) : 1.0f;  // m = -inf: 0
          if (moves) m[r] = high - 6.0f;
          l[r] *= shrink[r];
        }
        together();  // before the maxima are written again
        if (i > 0) {
          // (scores of tile c complete after the sum of tile c - 2, so this barrier is at most one phase behind)
          wait(&b.o[x ^ 1], ((c - 1) >> 1) & 1);
          if (any(!ok)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int y = 0; y < S::kUnits * kParts; ++y) {
            const uint32_t at = lanes + 128 + y / kParts * 64 + y % kParts * kRows;
            uint32_t o[16];
            tmem_ld16(o, at);
            tmem_wait_ld();
            settle16(o);
#pragma unroll
            for (int r = 0; r < kRows; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * shrink[r]);
            tmem_st16(at, o);
          }
          tmem_wait_st();
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; r += 4) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = ex2(s[r + k] - (m[r + k] == -INFINITY ? 0.0f : m[r + k]));
          l[r + k] = fmaf(w[k], e.z, l[r + k]);
        }
        uint32_t part[kParts];
        parts4(w[0], w[1], w[2], w[3], part);
#pragma unroll
        for (int y = 0; y < kParts; ++y)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int n = y * kRows + r + k;
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(weights + x * kOperandBytes + n * 128 + (((tid >> 4) ^ (n & 7)) << 4) + (tid & 15)),
                         "r"(part[y] >> (8 * k))
                         : "memory");
          }
      }
      fence_proxy_async_smem();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.p[x]);
      __syncwarp();
    }
    if (!ok) break;
    const uint32_t end = g + nt - 1;
    // every score of the item is computed: its queries may go
    const bool more = walk.next(p, later);
    if (more) fetch(later);
    g += nt;
    // sums of the weights over the keys: of a warp, then of all
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      l[r] = warp_sum(l[r]);
      if (lane == r) sh.top[warp][r] = l[r];
    }
    together();
#pragma unroll
    for (int r = 0; r < kRows; ++r) l[r] = (sh.top[0][r] + sh.top[1][r]) + (sh.top[2][r] + sh.top[3][r]);
    together();  // (also: what the rows see has been read)
    if (more) queries_loaded(later);
    wait(&b.o[end & 1], (end >> 1) & 1);  // one that ran out leaves the outputs incomplete; the next item's first vote ends the loop
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
    const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * S::kRows;
#pragma unroll 1
    for (int u = 0; u < S::kUnits; ++u) {
      float o[kRows];
      load_rows(lanes + 128 + u * 64, o);
      const int d = u * 128 + tid;
      if (d < p.head_dim) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r >= rows) break;
          if (whole) {
            const int t = (row0 + r) / p.group, head = it.h * (int)p.group.d + row0 + r - t * (int)p.group.d;
            st_u16(static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs + d,
                   round1<DT>(l[r] == 0.0f ? 0.0f : o[r] / l[r]));  // a row that saw nothing gives 0
          } else {
            p.part_o[(at + r) * p.part_dim + d] = o[r];
          }
        }
      }
      __syncwarp();
    }
    if (warp == 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (lane == r && r < rows) {
          if (!whole) {
            *reinterpret_cast<float2*>(p.part_ml + (at + r) * 2) = make_float2(m[r], l[r]);
          } else if (p.lse) {
            const int t = (row0 + r) / p.group, head = it.h * (int)p.group.d + row0 + r - t * (int)p.group.d;
            p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l[r] == 0.0f ? -INFINITY : (m[r] + log2f(l[r])) * 0.69314718055994531f;
          }
        }
    }
    if (it.first && !it.last) {
      goes_on = true;
      if (tid == 0) write_header(p, sh.span, &it);
    }
    it = later;
    have = more;
  }
  if (tid == 0 && !goes_on) write_header(p, sh.span, nullptr);
}

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 2) attn8_few(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                         const __grid_constant__ CUtensorMap vmap) {
  using S = Few<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ FewShared sh;
  Bars& b = sh.b;
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // swizzled tiles start on 1024 bytes
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostSlots; ++i) {
      mbar_init(&b.k.full[i], 1);
      mbar_init(&b.k.empty[i], 1);
      mbar_init(&b.v.full[i], 1);
      mbar_init(&b.v.empty[i], 1);
      b.k.issued[i] = b.v.issued[i] = 0;
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&b.s[x], 1);
      mbar_init(&b.o[x], 1);
      mbar_init(&b.p[x], 4);  // one arrival a warp
    }
    mbar_init(&b.q, 4);
    for (int x = 0; x < kScaleTiles; ++x) {
      mbar_init(&b.sc_full[x], 1);
      mbar_init(&b.sc_empty[x], 4);
    }
    mbar_init(&b.drain, 1);
    b.stop = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&b.tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&b.tmem);
  pdl_wait_and_release();
  find_span<S::kRows, kKeys, kThreads>(p, sh.span);

  const uint32_t queries = smem_addr(smem), weights = queries + S::kUnits * kOperandBytes, keys = weights + 2 * kOperandBytes,
                 values = keys + S::kKeySlots * kUnitBytes;
  if (warp < kMmaWarp) {
    few_softmax_role<DT, DP>(p, sh, queries, weights, tmem);
  } else if (warp == kLoadWarp) {
    load_role<S>(p, &kmap, sh.span, b, b.k, S::kKeySlots, keys, p.stall);
  } else if (warp == kLoadWarp + 1) {
    load_role<S>(p, &vmap, sh.span, b, b.v, S::kValueSlots, values, false);
    check_blocks(p);
  } else if (warp == kMmaWarp) {
    few_mma_role<DP>(p, sh, queries, weights, keys, values, tmem);
  } else {
    scale_role<S>(p, sh.span, b, sh.scales);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (b.stop && warp == kLoadWarp)  // copies in flight end before the CTA does
    for (int i = 0; i < kMostSlots; ++i) {
      if (b.k.issued[i] > (p.stall && i == 0 ? 1u : 0u)) mbar_wait_bounded(&b.k.full[i], (b.k.issued[i] - 1) & 1, p.wait_cycles);
      if (b.v.issued[i]) mbar_wait_bounded(&b.v.full[i], (b.v.issued[i] - 1) & 1, p.wait_cycles);
    }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int DT>
const void* few_of(int dp) {
  return dp == 256 ? reinterpret_cast<const void*>(&attn8_few<DT, 256>) : reinterpret_cast<const void*>(&attn8_few<DT, 128>);
}

}  // namespace

const void* attn8_few_kernel(bool bf16, int padded_dim) { return bf16 ? few_of<kBF16>(padded_dim) : few_of<kF16>(padded_dim); }

size_t attn8_few_smem(int padded_dim) { return (padded_dim == 256 ? Few<256>::kBytes : Few<128>::kBytes) + 1024; }

}  // namespace ar

// Paged attention over a cache of E4M3 codes on the fifth-generation tensor cores: rows on 16-byte boundaries,
// heads of a multiple of 16, pages of a multiple of 8 tokens.
//
// The division of the work, the roles of the warps and the tensor memory are those of the kernel for 16-bit
// caches.  What differs:
//
// Scores.  The keys' codes are operands of 8-bit matrix instructions as they are, which run at twice the 16-bit
// rate, so that q may be a sum of parts of 8 bits at the price of a 16-bit product:
//   x = hi + lo    bf16 (8 bits): hi = e4m3(x), lo = e5m2(x - hi);  fp16 (11 bits): hi + e4m3(x - hi) + e5m2(rest)
// E4M3 keeps 4 bits, with steps of 2^-9 at least, E5M2 3.  A row of q is scaled by a power of two, so that its
// largest element lies between 224 and 448: bf16 elements from 2^-6 on (fp16 from 2^-3) are then exact, smaller ones, whose
// rests of up to 2^-10 have more than 3 bits, off by up to 2^-14, 2^-21.8 of the largest.
//
// Values.  A warpgroup turns their codes to fp16, exactly, tile by tile, and the weights are fp16 too whatever
// the type of q (11 bits).  Parts of 8 bits for the weights as well, without that warpgroup, were slower: an
// element took 10 instructions in the softmax warps (4096 tokens over 28000: 854 us, 64 single tokens 260 us).
//
// Scales.  A row's weights take their keys' v scale, so that one reference serves both: with t_j = log2(vs_j),
//   w_j = 2^(s_j + t_j - m),  o = sum w_j c_j,  l = sum w_j / vs_j,  out = o / l,  lse = m + log2(l)
// and m kept so that the largest w of a row lies between 2^6 and 2^14, inside fp16's range.  Scales are the
// same for eight keys in a row at least; a warp of its own looks them up, tiles ahead, and leaves the k scale, t
// and 1 / vs of each eight keys of a tile in a ring in shared memory.
//
// Measured on GB300 with the joining kernel: 4096 tokens over 28000 (12 heads, 2 key heads of 128, bf16) 737 to 750 us,
// 1010 TFLOP/s (16-bit cache 510 to 530); in fp16 945 to 950 us (515), whose three parts of q leave the values one slot, so
// that none are on their way while a tile's are converted; 2 x 1024 tokens over 8000 (heads of 256) 258 us (154); six
// prompts of up to 1500 83 us (48); 17 requests, two of 700 tokens, window and cap 72 us (47).  The bound is the hand-over between the
// warps: 297 tiles an SM whose matrix instructions and softmax are left out still take 445 us, with the matrix
// instructions 640, with the softmax and without the conversion 715.  What the 16-bit kernel has over it: a third less
// for a softmax warp to issue (scales), and no warps that convert beside it.
#include <cuda.h>

#include <type_traits>

#include "ar_attn.cuh"
#include "ar_attn8.cuh"
#include "ar_attn_tc.cuh"
#include "ar_e4m3.cuh"
#include "ar_staged.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kThreads = kAttn8Threads;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvertWarp = 12;  // kLoadWarp + 1: values; 11: scales; four warps convert
constexpr uint32_t kTmemCols = 512;
constexpr int kSoftmaxRegs = 176, kIssueRegs = 104, kConvertRegs = 56;  // of 128 a thread at launch
static_assert(2 * kSoftmaxRegs + kIssueRegs + kConvertRegs == 4 * 128, "the split uses what the launch has");
constexpr int kRoomBytes = 13 * kUnitBytes;  // queries, fp16 values, rings

// FEW: for batches of 17 to 64 rows a request: items of 128 rows leave half of the queries' room to the rings (64
// single tokens of 48 heads over up to 9000, before they had a kernel of their own: 302 us, with items of 128 rows 273).
template <int DT, int DP, bool FEW>
struct Shape {
  static constexpr int kRows = DP == 256 || FEW ? 128 : 256;  // rows of an item
  static constexpr bool kTurns = DP == 128;             // the warpgroups take an item of one half by turns, tile by tile
  static constexpr int kParts = DT == kBF16 ? 2 : 3;    // of an element of q
  static constexpr int kUnits = DP / 128;               // ring slots that a tile of keys or values takes
  static constexpr int kPartBytes = kUnits * kUnitBytes;   // one part of a half's queries
  static constexpr int kHalfBytes = kParts * kPartBytes;
  static constexpr int kQueryBytes = kRows / 128 * kHalfBytes;
  static constexpr int kWide = 2, kWideBytes = 2 * kUnitBytes;  // units of values in fp16, in column blocks of 64
  static constexpr int kSlots = (kRoomBytes - kQueryBytes - kWide * kWideBytes) / kUnitBytes;
  static constexpr int kKeySlots = (kSlots + 1) / 2, kValueSlots = kSlots / 2;
  // Where the sums of a row's quarters meet: in the second half's queries, which an item of few rows has no use for,
  // or in its own, when its scores are computed and before the next item's come.
  static constexpr int kMeet = kRows == 256 ? kHalfBytes : 0;
};

// As in the kernel for 16-bit caches; keys and values have rings of their own.
struct Bars {
  Ring k, v;                     // keys are released by the matrix instructions, values by the four warps that convert
  uint64_t w_full[2], w_empty[2];  // values in fp16
  uint64_t q[2];
  uint64_t s[4], s2[4];          // scores of the first and second 64 keys
  uint64_t p[4], p2[4];
  uint64_t o[4];
  uint64_t half[4];              // first half of a tile's product complete (as p)
  uint64_t join[2];
  uint64_t meet[2];              // of a warpgroup's four warps, by quarters
  uint64_t sc_full[kScaleTiles], sc_empty[kScaleTiles];  // released by 8 warps, or twice by each of 4
  uint64_t drain;
  uint32_t tmem;
  int stop;
};

// ---- tcgen05 --------------------------------------------------------------------

__device__ __forceinline__ void mma_16bit(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptors, fp32 accumulator, 128 rows: scores of n keys, A in E4M3 or E5M2, B in E4M3; weighted
// sums of n columns, A and B in fp16, B's rows along the reduction.
__device__ __forceinline__ uint32_t scores_desc(int n, bool a_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ uint32_t sums_desc(int n) { return (1u << 4) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }

__device__ __forceinline__ void load_columns(uint32_t addr, float (&s)[64]) { load_scores(addr, s); }
__device__ __forceinline__ void load_columns(uint32_t addr, float (&s)[32]) {
  uint32_t r[32];
  tmem_ld32(r, addr);
  tmem_wait_ld();
  settle(r);
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(r[j]);
}

// ---- roles --------------------------------------------------------------------

// Every role walks the CTA's items for itself and counts barrier phases the same way (n, items, pairs, d, g as in
// the kernel for 16-bit caches; tiles: all so far, for the ring of scales).

// Items of no more than 32 rows: the rows are laid out four times, a warp's lanes each, and a warp takes 32 of a
// tile's 128 keys, so that the tile's softmax runs on all four sub-cores at once and takes a quarter of the time.
template <class S>
__device__ __forceinline__ bool by_quarters(const Item& it) {
  return S::kTurns && it.rows - it.qt * S::kRows <= 32;
}

template <class S>
__device__ __forceinline__ bool single_half(const Item& it) {
  return S::kRows == 128 || it.rows - it.qt * S::kRows <= 128;
}

// Values to fp16: a thread a key, 16 elements at a time.  Both layouts have 128-byte rows in 128-byte swizzle, so
// that eight rows' 16 bytes fall into different banks.  Keys that no row of the item sees become zeros: behind the
// request's end and in blocks that have left every row's window the cache holds anything, and a weight of 0 does not
// cancel a NaN.
template <class S>
__device__ void convert_role(const AttnParams& p, const SpanShared& span, Bars& b, uint32_t values, uint32_t wide) {
  const int lane = threadIdx.x & 31, row = (int)threadIdx.x - kConvertWarp * 32;
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t n = 0, slot = 0, round = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    const KeyRange seen = tile_keys<S::kRows>(p, it.q, it.qt);
    for (int t = 0; ok && t < nt; ++t) {
      const int key0 = it.range.tile(it.begin + t) * kKeys;
      const int lo = seen.low - key0, hi = seen.high - key0, pre = it.q.prefix - key0;
      const bool there = row < pre || (row < hi && row >= lo);
      for (int u = 0; u < S::kUnits; ++u, ++n) {
        const int chunks = min((p.head_dim - u * 128 + 15) / 16, 8);  // may be negative
        const uint32_t to = n & 1;
        ok = wait_for(&b.v.full[slot], round & 1, b, p) && wait_for(&b.w_empty[to], ((n >> 1) & 1) ^ 1, b, p);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t src = values + slot * kUnitBytes + row * 128, dst = wide + to * S::kWideBytes + row * 128;
        uint32_t in[8][4];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < chunks)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(in[c][0]), "=r"(in[c][1]), "=r"(in[c][2]), "=r"(in[c][3])
                         : "r"(src + ((c ^ (row & 7)) << 4))
                         : "memory");
        if (!there)
#pragma unroll
          for (int c = 0; c < 8; ++c) in[c][0] = in[c][1] = in[c][2] = in[c][3] = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c >= chunks) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
                  : "=r"(f[2 * i]), "=r"(f[2 * i + 1])
                  : "r"(in[c][half * 2 + i]));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + c / 4 * kUnitBytes + (((c % 4 * 2 + half) ^ (row & 7)) << 4)), "r"(f[0]),
                         "r"(f[1]), "r"(f[2]), "r"(f[3])
                         : "memory");
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&b.v.empty[slot]);
          mbar_arrive(&b.w_full[to]);
        }
        if (++slot == S::kValueSlots) {
          slot = 0;
          ++round;
        }
      }
    }
  }
}

template <class S>
__device__ void mma_role(const AttnParams& p, const SpanShared& span, Bars& b, uint32_t queries, uint32_t keys, uint32_t wide, uint32_t tmem) {
  const int ksteps = (p.head_dim + 31) / 32;
  // descriptors differ in the address alone, in units of 16 bytes: constant offsets are added
  const uint64_t q_desc = matrix_desc(queries, 16), k_desc = matrix_desc(keys, 16), v_desc = matrix_desc(wide, kUnitBytes);
  const bool one = elect_one();
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t slot = 0, round = 0, n = 0;  // of the unit of keys in turn; unit of values in turn
  uint32_t items = 0, pairs = 0, d = 0, g = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  auto wait_keys = [&] { return wait(&b.k.full[slot], round & 1); };
  auto release_keys = [&] {
    if (one) mma_commit(&b.k.empty[slot]);
    if (++slot == S::kKeySlots) {
      slot = 0;
      ++round;
    }
  };
  auto wait_values = [&](int u) { return wait(&b.w_full[(n + u) & 1], ((n + u) >> 1) & 1); };
  // queries of half h, part by part, times `count` keys of those in turn from key0 on (column part u of the head)
  // into score buffer `buf`
  auto scores = [&](int buf, int h, int u, int key0, int count) {
    const uint32_t idesc = scores_desc(count, false), idesc_last = scores_desc(count, true);
    const uint64_t k = k_desc + (slot * kUnitBytes + key0 * 128) / 16;
#pragma unroll
    for (int x = 0; x < S::kParts; ++x) {
      const uint64_t a = q_desc + (h * S::kHalfBytes + x * S::kPartBytes + u * kUnitBytes) / 16;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (u * 4 + s < ksteps) mma_8bit(tmem + buf * 128 + key0, a + s * 2, k + s * 2, x == S::kParts - 1 ? idesc_last : idesc, u > 0 || x > 0 || s > 0);
    }
  };
  // half `part` of the tile's weights in score buffer `buf` times the values in turn (column part u), to columns `to`
  auto weighted = [&](int buf, int u, int part, uint32_t to, bool more) {
    const uint64_t v = v_desc + ((n + u) & 1) * (S::kWideBytes / 16);
    const int cols = p.head_dim - u * 128;
    if (cols <= 0) return;
    const uint32_t idesc_o = sums_desc(cols < 128 ? cols : 128);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = part * 4 + s;
      mma_16bit(tmem + to + u * 128, tmem + buf * 128 + part * 64 + s * 8, v + ((k * 16 * 128) >> 4), idesc_o, more || k > 0);
    }
  };
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    if (single_half<S>(it)) {
      if (!wait(&b.q[0], items & 1)) break;
      for (int i = -1; ok && i < nt; ++i) {
        if (i + 1 < nt) {
          const uint32_t x = (g + i + 1) & 1;
          for (int u = 0; u < S::kUnits; ++u) {
            if (!wait_keys()) break;
            if (one) scores(x, 0, u, 0, kKeys);
            release_keys();
          }
          if (!ok) break;
          if (one) {
            mma_commit(&b.s[2 + x]);
            mma_commit(&b.s2[2 + x]);
          }
        }
        if (i < 0) continue;
        const uint32_t x = (g + i) & 1, phase = ((g + i) >> 1) & 1, sum_at = 256 + (S::kTurns ? x * 128 : 0);
        for (int u = 0; u < S::kUnits; ++u) wait_values(u);
        if (!wait(&b.p[2 + x], phase)) break;
        if (one) {
          for (int u = 0; u < S::kUnits; ++u) weighted(x, u, 0, sum_at, S::kTurns ? i > 1 : i > 0);
          mma_commit(&b.half[2 + x]);
        }
        if (!wait(&b.p2[2 + x], phase)) break;
        for (int u = 0; u < S::kUnits; ++u) {
          if (one) weighted(x, u, 1, sum_at, true);
          if (one) mma_commit(&b.w_empty[(n + u) & 1]);
        }
        n += S::kUnits;
        if (!ok) break;
        if (one) mma_commit(&b.o[2 + x]);
      }
      g += nt;
    } else {
      // Two halves take turns, 64 keys at a time: as soon as the weights of a half's 64 keys are used, the next
      // tile's scores take their columns, so that a half's softmax finds them when it is done with the other 64.
      if (!wait_keys()) break;
      for (int h = 0; ok && h < 2; ++h) {
        if (!wait(&b.q[h], (h ? pairs : items) & 1)) break;
        if (one) {
          scores(h, h, 0, 0, kKeys);
          mma_commit(&b.s[h]);
          mma_commit(&b.s2[h]);
        }
      }
      if (!ok) break;
      release_keys();
      for (int i = 0; ok && i < nt; ++i, ++d) {
        const bool more = i + 1 < nt;
        if (!wait_values(0)) break;
        for (int h = 0; ok && h < 2; ++h) {
          if (!wait(&b.p[h], d & 1)) break;
          if (one) {
            weighted(h, 0, 0, 256 + h * 128, i > 0);
            mma_commit(&b.half[h]);
          }
          if (!more) continue;
          if (h == 0 && !wait_keys()) break;
          if (one) {
            scores(h, h, 0, 0, 64);
            mma_commit(&b.s[h]);
          }
        }
        for (int h = 0; ok && h < 2; ++h) {
          if (!wait(&b.p2[h], d & 1)) break;
          if (one) {
            weighted(h, 0, 1, 256 + h * 128, true);
            mma_commit(&b.o[h]);
            if (h == 1) mma_commit(&b.w_empty[n & 1]);
            if (more) {
              scores(h, h, 0, 64, 64);
              mma_commit(&b.s2[h]);
            }
          }
        }
        if (!ok) break;
        ++n;
        if (more) release_keys();
      }
      ++pairs;
    }
    ++items;
  }
  if (!ok) {  // matrix instructions in flight end before tensor memory is freed
    if (one) mma_commit(&b.drain);
    mbar_wait_bounded(&b.drain, 0, p.wait_cycles);
  }
}

template <class S>
struct SoftmaxState {  // of a warp
  Walk<S::kRows, kKeys> walk;
  Item it, later;
};

// Shared by the softmax warps: what a row of q was divided by, of an item and the next (whose queries may come
// before the other warpgroup has looked); maxima and sums to join.
struct RowShared {
  float factor[2][256];
  float2 ml[256];
  float inv[2][32];  // of an item by quarters: reciprocals of the sums
};

template <class S, int DT, int DP, int EXT>
__device__ void softmax_role(const AttnParams& p, const SpanShared& span, SoftmaxState<S>& state, Bars& b, RowShared& rs,
                             const float4 (*scale_ring)[kScaleGroups], uint32_t queries, uint32_t tmem) {
  const int h = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
  // A thread's scores take most of its registers: what is the same for a warp stays in shared
  // memory.  Lane 0 alone steps the walk (a step reads and writes it), between two barriers of the warp.
  auto& walk = state.walk;
  Item &it = state.it, &later = state.later;
  if (lane == 0) walk.start(span);
  uint32_t d = 0, g = 0, joined = 0, met = 0, tiles = 0, items = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  auto arrive = [&](uint64_t* bar) {  // a warp's stores are done
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();  // tensor memory is read and written by whole warps
  };
  auto next_item = [&](Item& to) {  // the next one that this warpgroup has a part in
    __syncwarp();
    bool found = false;
    if (lane == 0) found = (S::kTurns || h == 0) && walk.next(p, to);
    __syncwarp();
    return __shfl_sync(0xffffffffu, found, 0) != 0;
  };
  // Queries: a warp loads, scales and splits the rows that its own lanes serve, 16 bytes a lane.  The first rows
  // are asked for while the last product of the item before still runs.  Columns beyond the head are zero.  Rows
  // beyond the item's keep what was there: they meet no other row, and nothing of them is stored.
  constexpr int kRowLanes = DP / 8, kStep = 32 / kRowLanes;  // lanes of a row, rows of a round of loads
  constexpr int kAhead = 4;                                  // rounds in flight
  const int col = (lane % kRowLanes) * 8, sub = lane / kRowLanes;
  uint4 raw[kAhead];
  bool loading = false;
  auto first_row = [&](const Item& it) { return it.qt * S::kRows + (by_quarters<S>(it) ? 0 : h * 128 + warp * 32); };
  auto warp_rows = [&](const Item& it) { return min(it.rows - first_row(it), 32); };
  auto fetch = [&](const Item& it, int r0) {
    const int base = first_row(it), rows = warp_rows(it);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)it.q.q0 * p.q_ts + (int64_t)it.h * (int)p.group.d * p.q_hs;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = r0 + k * kStep + sub;
      raw[k] = make_uint4(0, 0, 0, 0);
      if (r < rows && col < p.head_dim) {
        const int t = (base + r) / p.group, e = base + r - t * (int)p.group.d;
        raw[k] = ld_keep(q + t * p.q_ts + e * p.q_hs + col);
      }
    }
  };
  auto load_queries = [&](const Item& it) {
    if (h == 1 && single_half<S>(it)) return;
    loading = true;
    fetch(it, 0);
  };
  auto queries_loaded = [&](const Item& it, uint32_t item) {
    if (!loading) return;
    loading = false;
    const int rows = warp_rows(it);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kAhead * kStep) {
      if (r0) fetch(it, r0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * kStep + sub;
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
        uint32_t lo[S::kParts], hi[S::kParts];
        split4(f[0], f[1], f[2], f[3], lo);
        split4(f[4], f[5], f[6], f[7], hi);
        if (r < rows) {
          const int row = warp * 32 + r;
          const uint32_t dst = queries + h * S::kHalfBytes + (col >> 7) * kUnitBytes + row * 128 + ((((col & 127) >> 4) ^ (row & 7)) << 4) + (col & 8);
#pragma unroll
          for (int x = 0; x < S::kParts; ++x) sts_v2(dst + x * S::kPartBytes, lo[x], hi[x]);
          if (col == 0) rs.factor[item & 1][h * 128 + row] = __uint_as_float((unsigned)e << 23);
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.q[h]);
  };
  bool goes_on = false;
  bool have = next_item(it);
  if (have) load_queries(it);
  queries_loaded(it, items);
  while (have) {
    const int nt = it.end - it.begin;
    const bool one = single_half<S>(it);
    const bool turns = S::kTurns && one;
    const uint32_t to = lanes + 256 + (one && !S::kTurns ? 0 : h * 128);
    const bool quarters = by_quarters<S>(it);
    const int half_row = (one ? 0 : h * 128) + tid, row = it.qt * S::kRows + (quarters ? lane : half_row);
    const bool busy = row - lane < it.rows;  // the warp has a row
    RowView view = row_view(p, it, row);
    if (row >= it.rows) {  // no row: sees all, so that the warp need not mask for it; nothing of it is stored
      view.see_lo = 0;
      view.see_hi = 0x7fffffff;
    }
    float m = -INFINITY, factor = 1.0f;  // of the scores: what q was divided by (and what turns the product to log2 units)
    bool factor_known = false;
    uint64_t sum[4] = {0, 0, 0, 0};  // of the weights over their v scales, eight floats: one chain of additions would take longer than the exponentials
    const int first = turns ? (g ^ h) & 1 : 0, step = turns ? 2 : 1;
    for (int i = first; i < nt; i += step) {
      const uint32_t c = g + i, buf = one ? (c & 1) : h, x = one ? 2 + buf : h, phase = one ? (c >> 1) & 1 : (d + i) & 1;
      const uint32_t ts = lanes + buf * 128, at = tiles + i, stage = at % kScaleTiles;
      if (!wait(&b.s[x], phase)) break;
      if (!busy) {
        arrive(&b.p[x]);
        // not before: the tile before's second weights may still be on their way, and this arrival would count for them
        if (!wait(&b.s2[x], phase)) break;
        arrive(&b.p2[x]);
        if (lane == 0) mbar_arrive_count(&b.sc_empty[stage], one ? 2 : 1);
        continue;
      }
      if (!factor_known) {  // scores are there, so the queries were, and the row's factor with them
        factor_known = true;
        factor = rs.factor[items & 1][half_row];
        // within these bounds products of 0 stay 0, and what a k scale can add stays finite
        if (!EXT) factor = fminf(fmaxf(factor * p.scale_log2, 0x1p-90f), 0x1p95f);
      }
      if (!wait(&b.sc_full[stage], (at / kScaleTiles) & 1)) break;
      const uint32_t sc = smem_addr(scale_ring[stage]);
      auto key_scale = [&](int group) {  // and log2 of the v scale
        float2 e;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(e.x), "=f"(e.y) : "r"(sc + group * 16));
        return e;
      };
      auto all_scales = [&](int group) {
        float4 e;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(e.x), "=f"(e.y), "=f"(e.z), "=f"(e.w) : "r"(sc + group * 16));
        return e;
      };
      const int key0 = it.range.tile(it.begin + i) * kKeys, prefix = it.q.prefix;
      const bool edge = !__all_sync(0xffffffffu, (key0 + kKeys <= view.see_hi && key0 >= view.see_lo) || key0 + kKeys <= prefix);
      // `count` keys from column `col` on: maximum and weights from the same registers.  `second`: of the second 64 keys
      // of a tile whose first are on their way.  Weights of two keys a column.
      auto weights = [&](auto count, int col, bool second, auto& w) {
        constexpr int N = decltype(count)::value;
        float s[N];
        load_columns(ts + col, s);
        if constexpr (EXT != 0) {  // to products of q and k
#pragma unroll
          for (int j = 0; j < N; j += 8) {
            const float f = finite_product(key_scale((col + j) / 8).x, factor);
#pragma unroll
            for (int k = 0; k < 8; ++k) s[j + k] *= f;
          }
        }
        if (EXT || edge) shape_scores<EXT>(p, prefix, view, key0 + col, edge, s);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < N; j += 8) {
          const float2 e = key_scale((col + j) / 8);
          const float high = fmaxf(max3(max3(max3(s[j], s[j + 1], s[j + 2]), s[j + 3], s[j + 4]), s[j + 5], s[j + 6]), s[j + 7]);
          top[j / 8 % 4] = fmaxf(top[j / 8 % 4], EXT ? high + e.y : fmaf(high, e.x * factor, e.y));
        }
        const float high = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        const bool grown = high > m + 14.0f;  // m = -inf: any finite score
        if (__any_sync(0xffffffffu, grown)) {
          const float shrink = grown ? ex2(m - (high - 6.0f)) : 1.0f;  // m = -inf: 0
          if (grown) m = high - 6.0f;
          if (i > first || second) {
            // The products so far have to be complete: of the tile's first 64 keys, or of the tile before (of this
            // warpgroup: by turns that is so once the scores are there).  Each barrier is at most one phase behind.
            if (second) {
              if (!wait(&b.half[x], phase)) return;
            } else if (!one) {
              if (!wait(&b.o[x], phase ^ 1)) return;
            } else if (!S::kTurns) {
              if (!wait(&b.o[2 + ((c - 1) & 1)], ((c - 1) >> 1) & 1)) return;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float lo, hi;
              untwo(sum[k], lo, hi);
              sum[k] = two(lo * shrink, hi * shrink);
            }
#pragma unroll 1
            for (int k = 0; k < p.head_dim; k += 16) {
              uint32_t o[16];
              tmem_ld16(o, to + k);
              tmem_wait_ld();
              settle16(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
              tmem_st16(to + k, o);
            }
            tmem_wait_st();
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {  // eight keys with the same scales
          const float4 e = all_scales(col / 8 + j);
          const uint64_t mul = two(e.x * factor, e.x * factor), add = two(e.y - base, e.y - base);
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const uint64_t v = two(s[j * 8 + k], s[j * 8 + k + 1]);
            untwo(EXT ? add2(v, add) : fma2(v, mul, add), f[k], f[k + 1]);
            f[k] = ex2(f[k]);
            f[k + 1] = ex2(f[k + 1]);
            // the second product's operand: fp16, whose 11 bits are no fewer than the type's
            w[j * 4 + k / 2] = pack2<kF16>(f[k], f[k + 1]);
          }
          // of the unrounded weights
          sum[j & 3] = fma2(add2(add2(two(f[0], f[1]), two(f[2], f[3])), add2(two(f[4], f[5]), two(f[6], f[7]))), two(e.z, e.z), sum[j & 3]);
        }
      };
      if (quarters) {
        uint32_t w[16], none[16];
        weights(std::integral_constant<int, 32>(), warp * 32, false, w);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 16; ++j) none[j] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // the other keys are the other warps'
          const uint32_t to = ts + (k & 2) * 32 + (k & 1) * 16;
          if (k == warp)
            tmem_st16(to, w);
          else
            tmem_st16(to, none);
        }
        tmem_wait_st();
        arrive(&b.p[x]);
        arrive(&b.p2[x]);
      } else {
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          if (part && !wait(&b.s2[x], phase)) break;
          uint32_t w[32];
          weights(std::integral_constant<int, 64>(), part * 64, part != 0, w);
          if (!ok) break;
          tmem_st32(ts + part * 64, w);
          tmem_wait_st();
          arrive(part ? &b.p2[x] : &b.p[x]);  // the second product starts on the first half of the keys
        }
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive_count(&b.sc_empty[stage], one ? 2 : 1);
    }
    if (!ok) break;
    const uint32_t end = g + nt - 1;  // the last tile
    const bool other_ends = turns && (end & 1) != h;
    // (by turns a tile's score buffer is its warpgroup's: two tiles of one have one of the other between them, so that
    // no barrier of the other's can be two phases behind)
    if (other_ends && (h == 0 || nt > 1 || quarters) && !wait(&b.s[2 + (end & 1)], (end >> 1) & 1)) break;
    // every score of the item is computed: its queries may go
    const bool more = next_item(later), shared = turns && (nt > 1 || quarters);
    if (more) load_queries(later);
    tiles += nt;
    if (!one) {
      d += nt;
      if (!wait(&b.o[h], (d - 1) & 1)) break;
    } else {
      g += nt;
      // (scores of the last tile are there, so the sum's barrier is at most one phase behind)
      if ((shared || !other_ends) && !wait(&b.o[2 + (end & 1)], (end >> 1) & 1)) break;
    }
    if (!shared) queries_loaded(later, items + 1);
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
    float lo, hi;
    untwo(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), lo, hi);
    float l = lo + hi, scale0 = 1.0f, scale1 = 1.0f;
    if (shared) {
      rs.ml[threadIdx.x] = make_float2(m, l);
      arrive(&b.join[0]);
      if (!wait(&b.join[0], joined & 1)) break;
      // Not before: the next item's scores would complete phases that the other warpgroup still waits for.
      // (By quarters the room where the sums meet is in use until the end.)
      if (!quarters || (S::kMeet && h == 0)) queries_loaded(later, items + 1);
      if (quarters) {
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, rs.ml[k * 32 + lane].x);
        auto by = [&](int k) { return rs.ml[k * 32 + lane].x == -INFINITY ? 0.0f : ex2(rs.ml[k * 32 + lane].x - most); };
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) l += rs.ml[k * 32 + lane].y * by(k);
        scale0 = by(warp);
        scale1 = by(4 + warp);
        m = most;
      } else {
        const float2 mine = make_float2(m, l), theirs = rs.ml[threadIdx.x ^ 128];
        m = fmaxf(m, theirs.x);
        const float a = m == -INFINITY ? 0.0f : ex2(mine.x - m), z = m == -INFINITY ? 0.0f : ex2(theirs.x - m);
        // in one order for both, so that they agree
        scale0 = h ? z : a;
        scale1 = h ? a : z;
        l = (h ? theirs.y : mine.y) * scale0 + (h ? mine.y : theirs.y) * scale1;
      }
    }
    if (quarters) {
      // The four warps' sums of a row meet in shared memory, 32 columns at a time; each warpgroup joins half of the
      // columns.  (A warpgroup without a tile has left nothing in its columns: scale 0.)
      const int rows = it.rows - it.qt * S::kRows, row0 = it.qt * S::kRows;
      const int64_t at0 = ((int64_t)blockIdx.x * 2 + slot) * S::kRows;
      const uint32_t room = queries + S::kMeet + h * 16384;
      if (warp == 0) {
        rs.inv[h][lane] = l == 0.0f ? 0.0f : 1.0f / l;
        if (h == 0 && lane < rows) {
          if (!whole) {
            *reinterpret_cast<float2*>(p.part_ml + (at0 + lane) * 2) = make_float2(m, l);
          } else if (p.lse) {
            const int t = row / p.group, head = it.h * (int)p.group.d + row - t * (int)p.group.d;
            p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
          }
        }
      }
#pragma unroll 1
      for (int col = h * 64; col < min(p.head_dim, h * 64 + 64); col += 32) {
        uint32_t o[32];
        float f[32];
        tmem_ld32(o, lanes + 256 + col);
        tmem_wait_ld();
        settle(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = scale0 == 0.0f ? 0.0f : __uint_as_float(o[j]) * scale0;
        tmem_ld32(o, lanes + 384 + col);
        tmem_wait_ld();
        settle(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] += scale1 == 0.0f ? 0.0f : __uint_as_float(o[j]) * scale1;
        if (lane < rows)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(room + warp * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4)), "f"(f[4 * j]),
                         "f"(f[4 * j + 1]), "f"(f[4 * j + 2]), "f"(f[4 * j + 3])
                         : "memory");
        arrive(&b.meet[h]);
        if (!wait(&b.meet[h], met++ & 1)) break;
        for (int k = tid; k < rows * 8; k += 128) {
          const int r = k >> 3, j = k & 7, e = col + j * 4;
          if (e >= p.head_dim) continue;
          float4 sum4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float4 v;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                         : "r"(room + y * 4096 + r * 128 + ((j ^ (r & 7)) << 4))
                         : "memory");
            sum4 = make_float4(sum4.x + v.x, sum4.y + v.y, sum4.z + v.z, sum4.w + v.w);
          }
          if (whole) {
            const int t = (row0 + r) / p.group, head = it.h * (int)p.group.d + row0 + r - t * (int)p.group.d;
            const float inv = rs.inv[h][r];
            st_v2(static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs + e,
                  make_uint2(pack2<DT>(sum4.x * inv, sum4.y * inv), pack2<DT>(sum4.z * inv, sum4.w * inv)));
          } else {
            *reinterpret_cast<float4*>(p.part_o + (at0 + r) * p.part_dim + e) = sum4;
          }
        }
        arrive(&b.meet[h]);
        if (!wait(&b.meet[h], met++ & 1)) break;
      }
    } else if (busy && (shared || !other_ends)) {
      const bool mine = row < it.rows;
      const int t = row / p.group, head = it.h * (int)p.group.d + row - t * (int)p.group.d;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw nothing gives 0
      uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs;
      const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * S::kRows + half_row;
      float* part = p.part_o + at * p.part_dim;
      // 32 columns at a time, one copy of the code.  Of a shared item each warpgroup joins half of the columns.
      const int col0 = shared ? h * (DP / 2) : 0, cols = min(p.head_dim, shared ? col0 + DP / 2 : DP);
#pragma unroll 1
      for (int col = col0; col < cols; col += 32) {
        uint32_t o[32];
        __syncwarp();  // lanes without a row come from the last round early
        float f[32];
        tmem_ld32(o, (shared ? lanes + 256 : to) + col);
        tmem_wait_ld();
        settle(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(o[j]);
        if (shared) {
          tmem_ld32(o, lanes + 384 + col);
          tmem_wait_ld();
          settle(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = f[j] * scale0 + __uint_as_float(o[j]) * scale1;
        }
        if (!mine) continue;
        if (p.wide) {  // whole sectors
#pragma unroll
          for (int j = 0; j < 32; j += 16) {
            if (col + j >= p.head_dim) break;
            uint32_t v[8];
            if (whole) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = pack2<DT>(f[j + 2 * e] * inv, f[j + 2 * e + 1] * inv);
              st_v8(out + col + j, v);
            } else {
#pragma unroll
              for (int x = 0; x < 16; x += 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(f[j + x + e]);
                st_v8(part + col + j + x, v);
              }
            }
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          if (col + j >= p.head_dim) break;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = f[j + e];
          if (whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= inv;
            st_v4(out + col + j, pack8<DT>(v));
          } else {
            *reinterpret_cast<float4*>(part + col + j) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(part + col + j + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      if (mine && !(shared && h == 1)) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
        else if (p.lse)
          p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      }
    }
    // neither sum nor the room of m and l is written again until both warpgroups have read them
    if (shared) {
      arrive(&b.join[1]);
      if (!wait(&b.join[1], joined++ & 1)) break;
      queries_loaded(later, items + 1);
    }
    if (it.first && !it.last) {
      goes_on = true;
      if (threadIdx.x == 0) write_header(p, span, &it);
    }
    __syncwarp();  // every lane is done with the item
    if (lane == 0) it = later;
    __syncwarp();
    have = more;
    ++items;
  }
  if (threadIdx.x == 0 && !goes_on) write_header(p, span, nullptr);
}

template <int DT, int DP, bool FEW, int EXT>
__global__ void __launch_bounds__(kThreads, 1) attn8_tma(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                         const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<DT, DP, FEW>;
  extern __shared__ uint8_t raw[];
  __shared__ SpanShared span;
  __shared__ Bars b;
  __shared__ SoftmaxState<S> states[8];
  __shared__ RowShared rows;
  __shared__ float4 scales[kScaleTiles][kScaleGroups];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // swizzled tiles start on 1024 bytes
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostSlots; ++i) {
      mbar_init(&b.k.full[i], 1);
      mbar_init(&b.k.empty[i], 1);
      mbar_init(&b.v.full[i], 1);
      mbar_init(&b.v.empty[i], 4);
      b.k.issued[i] = b.v.issued[i] = 0;
    }
    for (int x = 0; x < S::kWide; ++x) {
      mbar_init(&b.w_full[x], 4);
      mbar_init(&b.w_empty[x], 1);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(&b.s[x], 1);
      mbar_init(&b.s2[x], 1);
      mbar_init(&b.o[x], 1);
      mbar_init(&b.half[x], 1);
      mbar_init(&b.p[x], 4);  // one arrival a warp
      mbar_init(&b.p2[x], 4);
    }
    for (int h = 0; h < 2; ++h) mbar_init(&b.q[h], 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&b.join[x], 8);
      mbar_init(&b.meet[x], 4);
    }
    for (int x = 0; x < kScaleTiles; ++x) {
      mbar_init(&b.sc_full[x], 1);
      mbar_init(&b.sc_empty[x], 8);
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
  find_span<S::kRows, kKeys, kThreads>(p, span);

  const uint32_t queries = smem_addr(smem), wide = queries + S::kQueryBytes, keys = wide + S::kWide * S::kWideBytes,
                 values = keys + S::kKeySlots * kUnitBytes;
  if (warp >= kConvertWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    convert_role<S>(p, span, b, values, wide);
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kLoadWarp) {
      load_role<S>(p, &kmap, span, b, b.k, S::kKeySlots, keys, p.stall);
    } else if (warp == kLoadWarp + 1) {
      load_role<S>(p, &vmap, span, b, b.v, S::kValueSlots, values, false);
      check_blocks(p);
    } else if (warp == kMmaWarp) {
      mma_role<S>(p, span, b, queries, keys, wide, tmem);
    } else {
      scale_role<S>(p, span, b, scales);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<S, DT, DP, EXT>(p, span, states[warp], b, rows, scales, queries, tmem);
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

template <int DT, int DP, bool FEW>
const void* tma_of(int ext) {
  switch (ext) {
    case 0: return reinterpret_cast<const void*>(&attn8_tma<DT, DP, FEW, 0>);
    case kCap: return reinterpret_cast<const void*>(&attn8_tma<DT, DP, FEW, kCap>);
    case kBias: return reinterpret_cast<const void*>(&attn8_tma<DT, DP, FEW, kBias>);
    case kCap | kBias | kWide: return reinterpret_cast<const void*>(&attn8_tma<DT, DP, FEW, kCap | kBias | kWide>);
    default: return reinterpret_cast<const void*>(&attn8_tma<DT, DP, FEW, kCap | kBias>);
  }
}

template <int DT>
const void* tma_of(int dp, bool few, int ext) {
  return dp == 256 ? tma_of<DT, 256, false>(ext) : few ? tma_of<DT, 128, true>(ext) : tma_of<DT, 128, false>(ext);
}

}  // namespace

const void* attn8_tma_kernel(bool bf16, int padded_dim, bool few, float cap, bool bias) {
  const int ext = score_forms(cap, bias);
  return bf16 ? tma_of<kBF16>(padded_dim, few, ext) : tma_of<kF16>(padded_dim, few, ext);
}

size_t attn8_tma_smem() { return kRoomBytes + 1024; }

}  // namespace ar

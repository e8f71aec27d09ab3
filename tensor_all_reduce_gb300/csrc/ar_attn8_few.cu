// Paged attention over a cache of E4M3 codes for few rows a request (single tokens, drafts): the products turned
// around, so that keys and values, not queries, are the 128-row operand.
//
// An item is up to 8 (or 16) query rows of one request and key head.  With Q = hi + mid / 16 + lo / 256 in three
// E4M3 parts (14 bits) and weights in four, each of the rest of the one before times 32 (18 bits and more), side by side as
// columns, a tile of 128 keys is two products of 8-bit matrix instructions:
//   scores   S[key, (part, row)] = K[key, d] Q[(part, row), d]          128 x 32 (48) x head
//   sums     O[d, (part, row)]  += V[key, d]^T W[key, (part, row)]      128 x 32 (64) x 128, for each 128 of the head
// Each byte of keys and values is thus read from shared memory once, as it came, and the tensor core's time and
// the softmax's do not count 128 rows where there are six.  The kernel that keeps queries as the 128-row operand
// reads keys twice (two parts), turns values to fp16 and was bound by that traffic in shared memory: 64 single
// tokens over up to 9000 keys, 48 heads, 8 key heads of 128: 273 us.
//
// A thread of the softmax warpgroup owns a key: it adds up the parts of the key's scores, and its weights, times
// the v scale as in ar_attn8_tma.cu, go to shared memory as parts.  The references m of the rows are the same
// in all threads; they move only when some weight of a tile would exceed 2^8 (one vote a tile), and then so that
// the row's largest becomes 2^6.  The fourth part's steps are 2^-24, so that a weight is off by 2^-31 of the largest
// at most: many small ones under one that is 2^20 times each keep their sum.  (Three parts a factor of 16 apart held weights
// to 2^-24 of the largest: of 160000 equal ones that are 2^-20 of it the sum came out 1 % off, at 2^-24 10 to 20 %.)
// A key's row of weights lies along its parts and rows, 32 (64) bytes that its thread writes 16 at a time.  (As rows along
// the keys, a byte at a time, the fourth part took the 64 single tokens below from 169 to 189 us.)
//
// Measured on GB300 with the joining kernel (48 heads, 8 key heads of 128, bf16, pages of 16): the 64 tokens above 162 us,
// 4.2 TB/s (676 MB; over a 16-bit cache of twice the bytes 213 to 230 us); 12 rows a request 273,
// heads of 64 and 256 165 and 272.  The copies alone take 154 us: a row of 128 bytes lies 1 KB from the next one's,
// between the other heads' (where there is one key head 125 us).  The rest is a tile's way through the softmax's one
// warpgroup, whose instructions wait on each other and on their own fetching.  What it took from 209 us on: the vote
// looked at a tile later, references in shared memory, 8 rows where 16 are not needed, weights in rows of a key.
//
// Two CTAs an SM, 256 threads each: a warpgroup for the softmax; warps for the matrix instructions, keys, values
// and scales.  Work division, parts of split items and their joining are the other kernels'.  Every wait is bounded.
#include <cuda.h>

#include "ar_attn8.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kParts = 3, kWeightParts = 4;
constexpr int kThreads = 256;
constexpr int kMmaWarp = 4, kLoadWarp = 5;  // kLoadWarp + 1: values; the last: scales
constexpr uint32_t kTmemCols = 256;                         // two score buffers and two sums, 64 columns each
// A part holds the rest of the one before, times this: rests are at most 2^4 for queries (up to 448), 2^3 for weights (up to 256).
constexpr float kPart = 16.0f, kWeightPart = 32.0f;

// ROWS: 8 or 16 rows of an item.
template <int DP, int ROWS>
struct Few {
  static constexpr int kRows = ROWS;
  static constexpr int kScoreColumns = (kParts * ROWS + 15) / 16 * 16;  // what the matrix instructions take; those behind the parts hold anything
  static constexpr int kSumColumns = kWeightParts * ROWS;
  static constexpr int kQueryBytes = kScoreColumns * 128;  // of 128 elements: rows of 128 bytes
  static constexpr int kWeightBytes = kKeys * kSumColumns;  // a row is a key
  static constexpr int kUnits = DP / 128;
  // What two CTAs of an SM have room for.  (Boxes asked into L2 three or six tiles ahead besides: 207 -> 221, 227 us.)
  static constexpr int kKeySlots = 3, kValueSlots = DP == 128 && ROWS == 8 ? 3 : 2;
  static constexpr int kBytes = kUnits * kQueryBytes + 2 * kWeightBytes + (kKeySlots + kValueSlots) * kUnitBytes;
};

struct Bars {
  Ring k, v;
  uint64_t q;          // queries stored
  uint64_t s[2];       // scores ready
  uint64_t p[2];       // weights stored
  uint64_t o[2];       // sum complete, of a tile
  uint64_t vote[2];    // a tile's scores have been looked at by the four softmax warps
  uint64_t meet;       // of these warps
  uint64_t sc_full[kScaleTiles], sc_empty[kScaleTiles];
  uint64_t drain;
  uint32_t tmem;
  int stop;
};

template <int ROWS>
struct FewShared {
  SpanShared span;
  Bars b;
  float4 scales[kScaleTiles][kScaleGroups];
  alignas(16) float factor[ROWS];  // of a row: what q was divided by
  int see_lo[ROWS], see_hi[ROWS], pos[ROWS];
  float slope[ROWS];
  alignas(16) float m[ROWS];        // what a row's weights refer to
  float top[4][ROWS];           // of a warp
  uint32_t grown[2];             // the last tile (counted from 1) whose scores outgrew the references
};

// The parts of four elements of a query.
__device__ __forceinline__ void parts4(float a, float b, float c, float d, uint32_t (&part)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    part[i] = codes4<false>(a, b, c, d);
    if (i + 1 == kParts) break;
    minus_codes4(part[i], a, b, c, d);
    a *= kPart, b *= kPart, c *= kPart, d *= kPart;
  }
}

// Instruction descriptors, fp32 accumulator, 128 rows, E4M3: scores; sums, both of whose operands have rows along the reduction.
__device__ __forceinline__ uint32_t scores_desc(int columns) { return (1u << 4) | ((uint32_t)(columns >> 3) << 17) | ((128u >> 4) << 24); }
__device__ __forceinline__ uint32_t sums_desc(int columns) { return scores_desc(columns) | (1u << 15) | (1u << 16); }

// Weights: a row of kSumColumns (32 or 64) bytes a key, eight rows after another, swizzled by as many bytes.
template <class S>
__device__ __forceinline__ uint64_t weights_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | ((uint64_t)(S::kSumColumns * 8 >> 4) << 32) | (1ull << 46) | ((S::kSumColumns == 32 ? 6ull : 4ull) << 61);
}

template <class S>
__device__ void few_mma_role(const AttnParams& p, FewShared<S::kRows>& sh, uint32_t queries, uint32_t weights, uint32_t keys, uint32_t values, uint32_t tmem) {
  Bars& b = sh.b;
  const int lane = threadIdx.x & 31;
  const int ksteps = (p.head_dim + 31) / 32;
  const uint32_t idesc_s = scores_desc(S::kScoreColumns), idesc_o = sums_desc(S::kSumColumns);
  const uint64_t q_desc = matrix_desc(queries, 16), w_desc = weights_desc<S>(weights), k_desc = matrix_desc(keys, 16), v_desc = matrix_desc(values, kUnitBytes);
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
        const uint64_t a = k_desc + ks * (kUnitBytes / 16), q = q_desc + u * (S::kQueryBytes / 16);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (u * 4 + s < ksteps) mma_8bit(tmem + x * 64, a + s * 2, q + s * 2, idesc_s, u > 0 || s > 0);
        mma_commit(&b.k.empty[ks]);
      }
      if (++ks == S::kKeySlots) ks = 0, ++kr;
    }
    if (one) mma_commit(&b.s[x]);
  };
  // Values of keys that no row of the item sees become zeros: in blocks that have left every row's window, and in the
  // last box behind the request's end (boxes behind it come as zeros), the cache holds anything, and a weight of 0 does
  // not cancel a NaN.
  KeyRange seen = {0, 0};
  auto has_unseen = [&](int key0) { return key0 + kKeys > it.q.prefix && (key0 + kKeys > seen.high || max(key0, it.q.prefix) < seen.low); };
  auto clear_unseen = [&](int key0) {
    const int pre = max(it.q.prefix - key0, 0), lo = min(seen.low - key0, kKeys), hi = min(max(seen.high - key0, 0), kKeys);
    const int end = min((max(it.q.len - key0, 0) + p.box_rows - 1) / p.box_rows * p.box_rows, kKeys);
    const uint32_t v = values + vs * kUnitBytes;
    for (int x = pre * 8 + lane; x < end * 8; x += 32)
      if (x < lo * 8 || x >= hi * 8) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + x * 16), "r"(0) : "memory");
    fence_proxy_async_smem();
    __syncwarp();
  };
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    seen = tile_keys<S::kRows>(p, it.q, it.qt);
    if (!wait(&b.q, items & 1)) break;
    scores(g & 1);
    for (int i = 0; ok && i < nt; ++i) {
      if (i + 1 < nt) scores((g + i + 1) & 1);
      if (!ok) break;
      const uint32_t x = (g + i) & 1;
      const int key0 = it.range.tile(it.begin + i) * kKeys;
      const bool unseen = has_unseen(key0);
      if (!wait(&b.p[x], ((g + i) >> 1) & 1)) break;
      for (int u = 0; u < S::kUnits; ++u) {
        if (!wait(&b.v.full[vs], vr & 1)) break;
        if (unseen) clear_unseen(key0);
        if (one) {
          const uint64_t a = v_desc + vs * (kUnitBytes / 16), w = w_desc + x * (S::kWeightBytes / 16);
          if (u * 128 < p.head_dim)
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_8bit(tmem + 128 + u * 64, a + ((s * 32 * 128) >> 4), w + ((s * 32 * S::kSumColumns) >> 4), idesc_o, i > 0 || s > 0);
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

// The parts of the rows in tensor memory, added up: of scores and of weighted sums.
__device__ __forceinline__ void load_scores(uint32_t addr, float (&f)[16]) {
  uint32_t a[32], c[16];
  tmem_ld32(a, addr);
  tmem_ld16(c, addr + 32);
  tmem_wait_ld();
  settle(a);
  settle16(c);
#pragma unroll
  for (int r = 0; r < 16; ++r) f[r] = fmaf(fmaf(__uint_as_float(c[r]), 1.0f / kPart, __uint_as_float(a[16 + r])), 1.0f / kPart, __uint_as_float(a[r]));
}
__device__ __forceinline__ void load_scores(uint32_t addr, float (&f)[8]) {
  uint32_t a[32];
  tmem_ld32(a, addr);
  tmem_wait_ld();
  settle(a);
#pragma unroll
  for (int r = 0; r < 8; ++r) f[r] = fmaf(fmaf(__uint_as_float(a[16 + r]), 1.0f / kPart, __uint_as_float(a[8 + r])), 1.0f / kPart, __uint_as_float(a[r]));
}
template <int ROWS>
__device__ __forceinline__ void load_sums(uint32_t addr, float (&f)[ROWS]) {
#pragma unroll
  for (int at = kWeightParts * ROWS - 32; at >= 0; at -= 32) {  // the last parts first
    uint32_t a[32];
    tmem_ld32(a, addr + at);
    tmem_wait_ld();
    settle(a);
#pragma unroll
    for (int y = 32 / ROWS - 1; y >= 0; --y)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float part = __uint_as_float(a[y * ROWS + r]);
        f[r] = at + y * ROWS == (kWeightParts - 1) * ROWS ? part : fmaf(f[r], 1.0f / kWeightPart, part);
      }
  }
}

template <int DT, int DP, class S>
__device__ void few_softmax_role(const AttnParams& p, FewShared<S::kRows>& sh, uint32_t queries, uint32_t weights, uint32_t tmem) {
  constexpr int kRows = S::kRows;
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
  auto four = [](const float* x) {  // read anew at each use: kept in registers they spilled
    float4 f;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(smem_addr(x)) : "memory");
    return f;
  };
  uint32_t met = 0;
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  auto together = [&] {  // the four warps, with the others' bound
    arrive(&b.meet);
    return wait(&b.meet, met++ & 1);
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
        sts_v2(queries + (col >> 7) * S::kQueryBytes + n * 128 + ((((col & 127) >> 4) ^ (n & 7)) << 4) + (col & 8), lo[x], hi[x]);
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
        sh.m[r] = -INFINITY;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.q);
    return together();  // what the rows see is there for all
  };
  Item it = {}, later = {};
  bool have = walk.next(p, it);
  if (have) {
    fetch(it);
    have = queries_loaded(it);
  }
  while (have) {
    const int nt = it.end - it.begin, row0 = it.qt * S::kRows, rows = min(it.rows - row0, S::kRows);
    float l[kRows];
    int lo = 0, hi = 0x7fffffff;  // keys that all rows see
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      l[r] = 0.0f;
      lo = max(lo, sh.see_lo[r]);
      hi = min(hi, sh.see_hi[r]);
    }
    // A tile's scores in log2 units with log2 of the v scale, masked; e_z: 1 / v scale.  The warps say whether some
    // outgrow the references, and look at the answer a tile later, so that nobody waits for it.
    auto prepare = [&](int i, float (&s)[kRows], float& e_z) {
      const uint32_t c = g + i, x = c & 1, stage = c % kScaleTiles;
      if (!wait(&b.s[x], (c >> 1) & 1) || !wait(&b.sc_full[stage], (c / kScaleTiles) & 1)) return;
      const float4 e = sh.scales[stage][tid >> 3];
      arrive(&b.sc_empty[stage]);
      e_z = e.z;
      load_scores(lanes + x * 64, s);
      const int key0 = it.range.tile(it.begin + i) * kKeys, key = key0 + tid, prefix = it.q.prefix;
      const bool edge = !((key0 + kKeys <= hi && key0 >= lo) || key0 + kKeys <= prefix);
      if (bent) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          RowView v;
          v.pos = sh.pos[r];
          v.slope = sh.slope[r];
          s[r] = bend(p, v, s[r] * finite_product(e.x, sh.factor[r]), key) + e.y;
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          const float4 f = four(&sh.factor[r]);
          s[r] = fmaf(s[r], f.x * e.x, e.y);
          s[r + 1] = fmaf(s[r + 1], f.y * e.x, e.y);
          s[r + 2] = fmaf(s[r + 2], f.z * e.x, e.y);
          s[r + 3] = fmaf(s[r + 3], f.w * e.x, e.y);
        }
      }
      if (edge)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (!(key < prefix || (key < sh.see_hi[r] && key >= sh.see_lo[r]))) s[r] = -INFINITY;
      bool grown = false;
#pragma unroll
      for (int r = 0; r < kRows; r += 4) {
        const float4 m = four(&sh.m[r]);  // -inf: any finite score
        grown = grown || s[r] > m.x + 8.0f || s[r + 1] > m.y + 8.0f || s[r + 2] > m.z + 8.0f || s[r + 3] > m.w + 8.0f;
      }
      if (grown) *reinterpret_cast<volatile uint32_t*>(&sh.grown[x]) = c + 1;
      arrive(&b.vote[x]);
    };
    float s[kRows], e_z = 1.0f;
    prepare(0, s, e_z);
    for (int i = 0; ok && i < nt; ++i) {
      const uint32_t c = g + i, x = c & 1;
      if (!wait(&b.vote[x], (c >> 1) & 1)) break;
      if (*reinterpret_cast<volatile uint32_t*>(&sh.grown[x]) == c + 1) {
        float shrink[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float top = s[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (lane == r) sh.top[warp][r] = top;
        }
        if (!together()) break;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float high = fmaxf(fmaxf(sh.top[0][r], sh.top[1][r]), fmaxf(sh.top[2][r], sh.top[3][r]));
          const float m = sh.m[r];
          const bool moves = high > m + 8.0f;
          shrink[r] = moves ? ex2(m - (high - 6.0f)) : 1.0f;  // m = -inf: 0
          l[r] *= shrink[r];
        }
        if (!together()) break;  // every warp has read the maxima and references
        if (warp == 0 && lane < kRows) {
          const float high = fmaxf(fmaxf(sh.top[0][lane], sh.top[1][lane]), fmaxf(sh.top[2][lane], sh.top[3][lane]));
          if (high > sh.m[lane] + 8.0f) sh.m[lane] = high - 6.0f;
        }
        if (!together()) break;  // before the maxima are written again
        if (i > 0) {
          // (scores of tile c complete after the sum of tile c - 2, so this barrier is at most one phase behind)
          if (!wait(&b.o[x ^ 1], ((c - 1) >> 1) & 1)) break;
#pragma unroll 1
          for (int y = 0; y < S::kUnits * (S::kSumColumns / 16); ++y) {
            const uint32_t at = lanes + 128 + y / (S::kSumColumns / 16) * 64 + y % (S::kSumColumns / 16) * 16;
            uint32_t o[16];
            tmem_ld16(o, at);
            tmem_wait_ld();
            settle16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink[j % kRows]);
            tmem_st16(at, o);
          }
          tmem_wait_st();
        }
      }
      float w[kRows];
#pragma unroll
      for (int r = 0; r < kRows; r += 4) {
        const float4 m = four(&sh.m[r]);
        const float base[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[r + k] = ex2(s[r + k] - (base[k] == -INFINITY ? 0.0f : base[k]));
          l[r + k] = fmaf(w[r + k], e_z, l[r + k]);
        }
      }
      if (i + 1 < nt) prepare(i + 1, s, e_z);
      if (!ok) break;
      // the key's row, 16 bytes at a time: two parts of 8 rows, or one of 16
      const uint32_t row = weights + x * S::kWeightBytes + tid * S::kSumColumns;
#pragma unroll
      for (int chunk = 0; chunk < S::kSumColumns / 16; ++chunk) {
        uint32_t part[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k * 4 % kRows;
          part[k] = codes4<false>(w[r], w[r + 1], w[r + 2], w[r + 3]);
          if (chunk * 16 + k * 4 < (kWeightParts - 1) * kRows) {
            minus_codes4(part[k], w[r], w[r + 1], w[r + 2], w[r + 3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[r + e] *= kWeightPart;
          }
        }
        const int swizzle = S::kSumColumns == 32 ? (tid >> 2) & 1 : (tid >> 1) & 3;
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((chunk ^ swizzle) << 4)), "r"(part[0]), "r"(part[1]), "r"(part[2]), "r"(part[3])
                     : "memory");
      }
      fence_proxy_async_smem();
      fence_before();
      arrive(&b.p[x]);
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
    if (!together()) break;
#pragma unroll
    for (int r = 0; r < kRows; ++r) l[r] = (sh.top[0][r] + sh.top[1][r]) + (sh.top[2][r] + sh.top[3][r]);
    const float m = sh.m[lane % kRows];
    if (!together()) break;  // (also: what the rows see has been read)
    if (more && !queries_loaded(later)) break;
    if (!wait(&b.o[end & 1], (end >> 1) & 1)) break;
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
    const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * S::kRows;
#pragma unroll 1
    for (int u = 0; u < S::kUnits; ++u) {
      float o[kRows];
      load_sums(lanes + 128 + u * 64, o);
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
            *reinterpret_cast<float2*>(p.part_ml + (at + r) * 2) = make_float2(m, l[r]);
          } else if (p.lse) {
            const int t = (row0 + r) / p.group, head = it.h * (int)p.group.d + row0 + r - t * (int)p.group.d;
            p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l[r] == 0.0f ? -INFINITY : (m + log2f(l[r])) * 0.69314718055994531f;
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

template <int DT, int DP, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) attn8_few(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                         const __grid_constant__ CUtensorMap vmap) {
  using S = Few<DP, ROWS>;
  extern __shared__ uint8_t raw[];
  __shared__ FewShared<ROWS> sh;
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
      mbar_init(&b.vote[x], 4);
    }
    mbar_init(&b.q, 4);
    mbar_init(&b.meet, 4);
    sh.grown[0] = sh.grown[1] = 0;
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

  const uint32_t queries = smem_addr(smem), weights = queries + S::kUnits * S::kQueryBytes, keys = weights + 2 * S::kWeightBytes,
                 values = keys + S::kKeySlots * kUnitBytes;
  if (warp < kMmaWarp) {
    few_softmax_role<DT, DP, S>(p, sh, queries, weights, tmem);
  } else if (warp == kLoadWarp) {
    load_role<S>(p, &kmap, sh.span, b, b.k, S::kKeySlots, keys, p.stall);
  } else if (warp == kLoadWarp + 1) {
    load_role<S>(p, &vmap, sh.span, b, b.v, S::kValueSlots, values, false);
    check_blocks(p);
  } else if (warp == kMmaWarp) {
    few_mma_role<S>(p, sh, queries, weights, keys, values, tmem);
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

template <int DT, int ROWS>
const void* few_of(int dp) {
  return dp == 256 ? reinterpret_cast<const void*>(&attn8_few<DT, 256, ROWS>) : reinterpret_cast<const void*>(&attn8_few<DT, 128, ROWS>);
}

}  // namespace

const void* attn8_few_kernel(bool bf16, int padded_dim, int rows) {
  if (rows == 8) return bf16 ? few_of<kBF16, 8>(padded_dim) : few_of<kF16, 8>(padded_dim);
  return bf16 ? few_of<kBF16, 16>(padded_dim) : few_of<kF16, 16>(padded_dim);
}

size_t attn8_few_smem(int padded_dim, int rows) {
  if (rows == 8) return (padded_dim == 256 ? Few<256, 8>::kBytes : Few<128, 8>::kBytes) + 1024;
  return (padded_dim == 256 ? Few<256, 16>::kBytes : Few<128, 16>::kBytes) + 1024;
}

}  // namespace ar

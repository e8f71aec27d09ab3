// Paged attention on the fifth-generation tensor cores: rows on 16-byte boundaries, pages of a
// multiple of 8 tokens.
//
// A CTA (one an SM, resident) takes items of 256 query rows (128 for heads of more than 128
// elements), in halves of 128, against tiles of 128 keys.  Of its twelve warps two load keys and
// values by TMA, box by box through the block table, into a ring of shared-memory slots; one
// issues the matrix instructions; a warpgroup for each half turns scores into weights (the last
// warp only completes the third warpgroup, which hands registers to the others).  A thread of a
// warpgroup owns one query row, so row maxima and sums need no exchange between threads.
//
// Tensor memory (512 columns of 128 lanes): two score buffers of 128 columns, and 256 columns for
// the weighted sums, 128 a half or all for one half.  The weights, 16-bit, take the first 64
// columns of their scores and are the second product's A operand from there, so they never touch
// shared memory.  Matrix instructions of one CTA run in the order in which they are issued.  With
// two halves, one half's softmax runs while the tensor core works on the other's products; with
// one (few rows, wide heads) the two buffers hold its present and next tile, and the warpgroups
// take tiles by turns, each with a maximum and a sum of its own, joined at the item's end (17
// requests, two of them 700 tokens, window and cap: 56 us with one warpgroup, 53 us with both;
// heads of more than 128 have no columns for a second sum).
//
// The running maximum that the weights refer to moves only when a row's maximum has grown by more
// than 2^8 (in weight), since the result does not depend on the reference: then the sum in
// tensor memory is scaled.  Weights are thus at most 2^8, far inside both 16-bit ranges.
//
// Measured on GB300 with the joining kernel: 64 single tokens over up to 9000 keys (48 heads, 8 key
// heads of 128, 1.4 GB) 213 to 220 us, 6.4 to 6.6 TB/s, where memory is the bound; 4096 tokens over 28000
// (12 heads, 2 key heads of 128) 510 to 530 us, 1430 to 1480 TFLOP/s, bound by shared memory, which feeds both
// operands of the scores and the values, and by the exponentials; heads of 256 928 TFLOP/s, since 128 rows of an item
// leave twice the reads of keys and values a product; short prompts by an item's start and end.
//
// Every wait is bounded; one that runs out leaves code 1 in the status word, and all roles stop.
// Shared memory is full to 64 bytes: 225 KB of tiles for heads of 65 to 128, and about 2 KB static.
#include <cuda.h>

#include "ar_attn.cuh"
#include "ar_attn_tc.cuh"
#include "ar_staged.cuh"
#include "ar_two.cuh"

namespace ar {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9;  // and kLoadWarp + 1
constexpr uint32_t kTmemCols = 512;
// 384 threads at 168 registers; the third warpgroup gives 80 a thread to the other two
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * 168, "the split uses what the launch has");

template <int DP>
struct Shape {
  static constexpr int kRows = DP == 256 ? 128 : 256;   // rows of an item
  static constexpr bool kTurns = DP <= 128;             // the warpgroups take an item of one half by turns, tile by tile
  static constexpr int kUnits = DP == 256 ? 2 : 1;      // ring slots that a tile of keys or values takes
  static constexpr int kBlocks = DP / 64 / kUnits;      // 64-element (128-byte) column blocks of a unit
  static constexpr int kBlockBytes = kKeys * 128;       // one column block of 128 rows
  static constexpr int kUnitBytes = kBlocks * kBlockBytes;
  static constexpr int kTileBytes = kUnits * kUnitBytes;
  static constexpr int kQueryBytes = kRows / 128 * kTileBytes;
  static constexpr int kSlots = DP == 64 ? 10 : 5;
  static constexpr int kBytes = kQueryBytes + kSlots * kUnitBytes;
};

// Score buffers and their barriers: 0 and 1 for two halves, 2 and 3 (in the same columns) for the
// turns of an item of one half.
struct Bars {
  uint64_t full[10], empty[10];  // ring slots
  uint64_t q[2];                 // queries of a half stored
  uint64_t s[4];                 // scores ready
  uint64_t p[4], p2[4];          // weights of the first and second 64 keys stored
  uint64_t o[4];                 // sum complete: of half 0, 1 (an item), of one half (a tile, by turns)
  uint64_t join[2];              // sums of an item taken by turns: both there, both read
  uint64_t drain;
  uint32_t issued[10];           // rounds whose copies were issued, a slot
  uint32_t tmem;
  int stop;
};

// ---- tcgen05, 16-bit operands -------------------------------------------------

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor: 16-bit operands, fp32 accumulator, 128 rows, n columns.
template <int DT>
__device__ __forceinline__ uint32_t instr_desc(int n, bool b_rows_along_k) {
  constexpr uint32_t type = DT == kBF16 ? 1 : 0;
  return (1u << 4) | (type << 7) | (type << 10) | ((b_rows_along_k ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// 16 bytes to shared memory, the last 16 - bytes of them zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---- roles --------------------------------------------------------------------

// Every role walks the CTA's items for itself and counts barrier phases the same way:
//   n: units loaded into the ring; items: items so far (phase of q[0], o[...] of paired halves);
//   pairs: items of two halves; d: tiles of such items; g: tiles of items of one half.
// An item of one half has two score buffers (by turns), so that the next tile's scores are computed
// while the softmax works on the present one; one of two halves has one buffer each.  For heads of
// up to 128 the turns are the warpgroups' too: each keeps a maximum and a sum of its own over every
// other tile, and the two are joined at the item's end.

template <int DP>
__device__ __forceinline__ bool single_half(const Item& it) {
  return Shape<DP>::kRows == 128 || it.rows - it.qt * Shape<DP>::kRows <= 128;
}

// Two warps load, one the keys and one the values: with small pages a tile is up to 32 copies, and
// issuing them is what takes the time.  The lanes look the blocks up, one elected lane issues.
template <int DP>
__device__ void load_role(const AttnParams& p, bool keys, const CUtensorMap* map, const SpanShared& span, Bars& b, uint32_t ring) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  const int boxes = kKeys / p.box_rows;
  const bool one = elect_one();
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t n = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    const bool ahead = single_half<DP>(it);  // scores run a tile ahead
    // block of this lane's box, and its place in the block
    int block = 0, place = 0;
    auto look_up = [&](int t) {
      const int key = it.range.tile(it.begin + t) * kKeys + lane * p.box_rows;
      block = -1;
      place = 0;
      if (lane < boxes && key < it.q.len) {
        const int j = key / p.page;
        place = key - j * (int)p.page.d;
        block = p.table[(int64_t)it.r * p.table_stride + j];
      }
    };
    look_up(0);
    for (int t = 0; ok && t < nt; ++t) {
      // ring units of the item: keys 0, then (values t, keys t + 1), or (keys t + 1, values t) where scores run ahead
      uint32_t i;
      if (keys)
        i = t == 0 ? 0 : (ahead ? 2 * t - 1 : 2 * t);
      else
        i = ahead && t + 1 < nt ? 2 * t + 2 : 2 * t + 1;
      i = n + i * S::kUnits;
      // outside the cache: the copy fills with zeros
      const int w = (unsigned)block < (unsigned)p.num_blocks ? block : (int)p.num_blocks, y = place;
      if (t + 1 < nt) look_up(t + 1);
      for (int u = 0; u < S::kUnits; ++u, ++i) {
        const uint32_t slot = i % S::kSlots, round = i / S::kSlots;
        ok = __all_sync(0xffffffffu, ok && wait_for(&b.empty[slot], (round & 1) ^ 1, b, p));
        if (!ok) break;
        if (one) {
          mbar_arrive_expect_tx(&b.full[slot], S::kUnitBytes);
          b.issued[slot] = round + 1;
        }
        const uint32_t dst = ring + slot * S::kUnitBytes;
        for (int x = 0; x < boxes; ++x) {
          const int wx = __shfl_sync(0xffffffffu, w, x), yx = __shfl_sync(0xffffffffu, y, x);
          if (one && !(p.stall && i == 0))
#pragma unroll
            for (int cb = 0; cb < S::kBlocks; ++cb)
              tma_4d(dst + cb * S::kBlockBytes + x * p.box_rows * 128, map, u * 128 + cb * 64, yx, it.h, wx, &b.full[slot]);
        }
      }
    }
    n += 2 * nt * S::kUnits;
  }
}

template <int DT, int DP>
__device__ void mma_role(const AttnParams& p, const SpanShared& span, Bars& b, uint32_t queries, uint32_t ring, uint32_t tmem) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  const int ksteps = (p.head_dim + 15) / 16;
  const uint32_t idesc_s = instr_desc<DT>(kKeys, false);
  // descriptors differ in the address alone, in units of 16 bytes: constant offsets are added
  const uint64_t q_desc = matrix_desc(queries, 16), k_desc = matrix_desc(ring, 16), v_desc = matrix_desc(ring, S::kBlockBytes);
  const bool one = elect_one();
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t n = 0, items = 0, pairs = 0, d = 0, g = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  auto wait_unit = [&](uint32_t i) { return wait(&b.full[i % S::kSlots], (i / S::kSlots) & 1); };
  // queries of half h times the keys of unit i (column part u of the head) into score buffer `buf`
  auto scores = [&](int buf, int h, uint32_t i, int u) {
    const uint64_t a = q_desc + (h * S::kTileBytes + u * S::kUnitBytes) / 16, k = k_desc + (i % S::kSlots) * (S::kUnitBytes / 16);
#pragma unroll
    for (int s = 0; s < S::kUnitBytes / kKeys / 32; ++s) {
      const uint64_t off = ((s >> 2) * S::kBlockBytes + (s & 3) * 32) >> 4;
      if (u * 8 + s < ksteps) mma_ss(tmem + buf * 128, a + off, k + off, idesc_s, u > 0 || s > 0);
    }
  };
  // half `part` of the tile's weights in score buffer `buf` times the values of unit i, to columns `to`
  auto weighted = [&](int buf, uint32_t i, int u, int part, uint32_t to, bool more) {
    const uint64_t v = v_desc + (i % S::kSlots) * (S::kUnitBytes / 16);
    const int cols = ksteps * 16 - u * 128;
    if (cols <= 0) return;
    const uint32_t idesc_o = instr_desc<DT>(cols < 128 ? cols : 128, true);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = part * 4 + s;
      mma_ts(tmem + to + u * 128, tmem + buf * 128 + k * 8, v + ((k * 16 * 128) >> 4), idesc_o, more || k > 0);
    }
  };
  // Values behind the request's end: whole boxes came as zeros, the rest of the last box holds
  // whatever the cache does.  Zeroed, because a weight of 0 does not cancel an infinity.
  auto clear_tail = [&](int t, uint32_t i) {
    const int left = it.q.len - it.range.tile(it.begin + t) * kKeys;
    if (left >= kKeys) return;
    const int lo = max(left, 0), hi = min((lo + p.box_rows - 1) / p.box_rows * p.box_rows, kKeys);
    const uint32_t v = ring + (i % S::kSlots) * S::kUnitBytes;
    for (int x = lo * 8 + lane; x < hi * 8; x += 32)
#pragma unroll
      for (int cb = 0; cb < S::kBlocks; ++cb)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + cb * S::kBlockBytes + x * 16), "r"(0) : "memory");
    fence_proxy_async_smem();
    __syncwarp();
  };
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    if (single_half<DP>(it)) {
      if (!wait(&b.q[0], items & 1)) break;
      for (int i = -1; ok && i < nt; ++i) {
        if (i + 1 < nt) {
          const uint32_t x = (g + i + 1) & 1;
          for (int u = 0; u < S::kUnits; ++u, ++n) {
            if (!wait_unit(n)) break;
            if (one) {
              scores(x, 0, n, u);
              mma_commit(&b.empty[n % S::kSlots]);
            }
          }
          if (!ok) break;
          if (one) mma_commit(&b.s[2 + x]);
        }
        if (i < 0) continue;
        const uint32_t x = (g + i) & 1, phase = ((g + i) >> 1) & 1, sum_at = 256 + (S::kTurns ? x * 128 : 0);
        for (int u = 0; u < S::kUnits; ++u, ++n) {
          if (!wait_unit(n)) break;
          clear_tail(i, n);
          if (u == 0 && !wait(&b.p[2 + x], phase)) break;
          if (one) weighted(x, n, u, 0, sum_at, S::kTurns ? i > 1 : i > 0);
          if (u == 0 && !wait(&b.p2[2 + x], phase)) break;
          if (one) {
            weighted(x, n, u, 1, sum_at, true);
            mma_commit(&b.empty[n % S::kSlots]);
          }
        }
        if (!ok) break;
        if (one) mma_commit(&b.o[2 + x]);
      }
      g += nt;
    } else {
      if (!wait_unit(n)) break;
      for (int h = 0; ok && h < 2; ++h) {
        if (!wait(&b.q[h], (h ? pairs : items) & 1)) break;
        if (one) {
          scores(h, h, n, 0);
          mma_commit(&b.s[h]);
        }
      }
      if (!ok) break;
      if (one) mma_commit(&b.empty[n % S::kSlots]);
      ++n;
      for (int i = 0; ok && i < nt; ++i, ++d) {
        const bool more = i + 1 < nt;
        if (!wait_unit(n)) break;
        clear_tail(i, n);
        for (int h = 0; h < 2; ++h) {
          if (!wait(&b.p[h], d & 1)) break;
          if (one) weighted(h, n, 0, 0, 256 + h * 128, i > 0);
          if (!wait(&b.p2[h], d & 1)) break;
          if (one) {
            weighted(h, n, 0, 1, 256 + h * 128, true);
            if (h == 1) mma_commit(&b.empty[n % S::kSlots]);
          }
          if (more) {
            if (h == 0 && !wait_unit(n + 1)) break;
            if (one) {
              scores(h, h, n + 1, 0);
              mma_commit(&b.s[h]);
            }
          } else if (one) {
            mma_commit(&b.o[h]);
          }
        }
        if (!ok) break;
        if (one && more) mma_commit(&b.empty[(n + 1) % S::kSlots]);
        n += more ? 2 : 1;
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

template <int DP>
struct SoftmaxState {  // of a warp
  Walk<Shape<DP>::kRows, kKeys> walk;
  Item it, later;
};

template <int DT, int DP, int EXT>
__device__ void softmax_role(const AttnParams& p, const SpanShared& span, SoftmaxState<DP>& state, Bars& b, uint8_t* queries, uint32_t tmem) {
  using S = Shape<DP>;
  const int h = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
  const float scale = EXT ? 1.0f : p.scale_log2;
  // A thread's scores take most of its registers: what is the same for a warp stays in shared
  // memory.  Lane 0 alone steps the walk (a step reads and writes it), between two barriers of the warp.
  auto& walk = state.walk;
  Item &it = state.it, &later = state.later;
  if (lane == 0) walk.start(span);
  uint32_t pairs = 0, d = 0, g = 0, joined = 0;
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
  // Queries, 16 bytes a thread, neighbours along a row, by asynchronous copies: all are in flight
  // at once and hold no registers.  Columns beyond the head are zero.  Rows beyond the item's keep
  // what was there: they meet no other row, and nothing of them is stored.
  bool loading = false;
  auto load_queries = [&](const Item& it) {
    if (h == 1 && single_half<DP>(it)) return;
    loading = true;
    const uint32_t dst = smem_addr(queries + h * S::kTileBytes);
    const int base = it.qt * S::kRows + h * 128, rows = min(it.rows - base, 128);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)it.q.q0 * p.q_ts + (int64_t)it.h * (int)p.group.d * p.q_hs;
#pragma unroll 4
    for (int x = tid; x < rows * (DP / 8); x += 128) {
      const int r = x / (DP / 8), c = x % (DP / 8);
      const int t = (base + r) / p.group, e = base + r - t * (int)p.group.d;
      const uint16_t* src = q + t * p.q_ts + e * p.q_hs + c * 8;
      cp_async16(dst + (c >> 3) * S::kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4), c * 8 < p.head_dim ? src : q, c * 8 < p.head_dim ? 16 : 0);
    }
  };
  auto queries_loaded = [&] {
    if (!loading) return;
    loading = false;
    cp_async_wait();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.q[h]);
  };
  bool goes_on = false;
  bool have = next_item(it);
  if (have) load_queries(it);
  queries_loaded();
  while (have) {
    const int nt = it.end - it.begin;
    const bool one = single_half<DP>(it);
    const bool turns = S::kTurns && one;
    const uint32_t to = lanes + 256 + (one && !S::kTurns ? 0 : h * 128);
    const int half_row = (one ? 0 : h * 128) + tid, row = it.qt * S::kRows + half_row;
    const bool busy = row - lane < it.rows;  // the warp has a row
    RowView view = row_view(p, it, row);
    if (row >= it.rows) {  // no row: sees all, so that the warp need not mask for it; nothing of it is stored
      view.see_lo = 0;
      view.see_hi = 0x7fffffff;
    }
    float m = -INFINITY;
    uint64_t sum[4] = {0, 0, 0, 0};  // of the weights, eight floats: one chain of additions would take longer than the exponentials
    const int first = turns ? (g ^ h) & 1 : 0, step = turns ? 2 : 1;
    for (int i = first; i < nt; i += step) {
      const uint32_t c = g + i, buf = one ? (c & 1) : h, x = one ? 2 + buf : h, phase = one ? (c >> 1) & 1 : (d + i) & 1;
      const uint32_t ts = lanes + buf * 128;
      if (!wait(&b.s[x], phase)) break;
      if (!busy) {
        arrive(&b.p[x]);
        arrive(&b.p2[x]);
        continue;
      }
      // Twice over the scores: for the maximum (bent and masked scores go back to tensor memory) and
      // for the weights, 64 at a time.  Kept in registers from one to the other they spilled
      // (decode of 64 requests 220 us so, 217 us read twice; prefix with bias 60 and 59 us).
      const int key0 = it.range.tile(it.begin + i) * kKeys, prefix = it.q.prefix;
      const bool edge = !__all_sync(0xffffffffu, (key0 + kKeys <= view.see_hi && key0 >= view.see_lo) || key0 + kKeys <= prefix);
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (!EXT && !edge) {
        uint32_t s[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(s[k], ts + k * 32);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          settle(s[k]);
#pragma unroll
          for (int j = 0; j < 32; j += 2) top[k] = max3(top[k], __uint_as_float(s[k][j]), __uint_as_float(s[k][j + 1]));
        }
      } else {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          float s[64];
          load_scores(ts + part * 64, s);
          shape_scores<EXT>(p, prefix, view, key0 + part * 64, edge, s);
          uint32_t back[32];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < 32; ++j) back[j] = __float_as_uint(s[k * 32 + j]);
            tmem_st32(ts + part * 64 + k * 32, back);
          }
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = max3(top[k], s[j + k], s[j + 4 + k]);
        }
        tmem_wait_st();
      }
      const float high = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale;
      const bool grown = high > m + 8.0f;  // m = -inf: any finite score
      if (__any_sync(0xffffffffu, grown)) {
        const float shrink = grown ? ex2(m - high) : 1.0f;  // m = -inf: 0
        if (grown) m = high;
        if (i > first) {
          // the sum holds this warpgroup's tiles so far: that is so once the scores are there, but for
          // one warpgroup with scores that run ahead, where a barrier says so.  (Scores of tile c
          // complete after the sum of tile c - 2, so this barrier is at most one phase behind.)
          if (!S::kTurns && !wait(&b.o[2 + ((c - 1) & 1)], ((c - 1) >> 1) & 1)) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, hi;
            untwo(sum[k], lo, hi);
            sum[k] = two(lo * shrink, hi * shrink);
          }
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(o, to + k * 32);
            tmem_wait_ld();
            settle(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
            tmem_st32(to + k * 32, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      const uint64_t scale2 = two(scale, scale), base2 = two(-base, -base);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float s[64];
        load_scores(ts + part * 64, s);
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float a, z;
          untwo(fma2(two(s[2 * j], s[2 * j + 1]), scale2, base2), a, z);
          a = ex2(a);
          z = ex2(z);
          sum[j & 3] = add2(sum[j & 3], two(a, z));  // of the unrounded weights
          // the second product's operand is 16-bit: half a step, relative, a weight (outputs are 1.2 to 1.4
          // times as far from the 64-bit ones as with weights of 32 bits, which would be two operands and two products)
          w[j] = pack2<DT>(a, z);
        }
        tmem_st32(ts + part * 32, w);
        tmem_wait_st();
        arrive(part ? &b.p2[x] : &b.p[x]);  // the second product starts on the first half of the keys
      }
    }
    if (!ok) break;
    const uint32_t end = g + nt - 1;  // the last tile
    const bool other_ends = turns && (end & 1) != h;
    if (other_ends && (h == 0 || nt > 1) && !wait(&b.s[2 + (end & 1)], (end >> 1) & 1)) break;
    // every score of the item is computed: its queries may go
    const bool more = next_item(later), shared = turns && nt > 1;
    if (more && !(shared && h == 1)) load_queries(later);
    if (!one) {
      d += nt;
      if (!wait(&b.o[h], pairs++ & 1)) break;
    } else {
      g += nt;
      // (scores of the last tile are there, so the sum's barrier is at most one phase behind)
      if ((shared || !other_ends) && !wait(&b.o[2 + (end & 1)], (end >> 1) & 1)) break;
    }
    if (!shared) queries_loaded();
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
    float lo, hi;
    untwo(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), lo, hi);
    float l = lo + hi, scale0 = 1.0f, scale1 = 1.0f;
    if (shared) {  // the second half's queries have no use for an item of one half: their room takes m and l
      float2* ml = reinterpret_cast<float2*>(queries + S::kTileBytes);
      ml[threadIdx.x] = make_float2(m, l);
      arrive(&b.join[0]);
      if (!wait(&b.join[0], joined & 1)) break;
      // Not before: the next item's scores would complete phases that the other warpgroup still waits for.
      queries_loaded();
      const float2 mine = make_float2(m, l), theirs = ml[threadIdx.x ^ 128];
      m = fmaxf(m, theirs.x);
      const float a = m == -INFINITY ? 0.0f : ex2(mine.x - m), z = m == -INFINITY ? 0.0f : ex2(theirs.x - m);
      // in one order for both, so that they agree
      scale0 = h ? z : a;
      scale1 = h ? a : z;
      l = (h ? theirs.y : mine.y) * scale0 + (h ? mine.y : theirs.y) * scale1;
    }
    if (busy && (shared || !other_ends)) {
      const bool mine = row < it.rows;
      const int t = row / p.group, head = it.h * (int)p.group.d + row - t * (int)p.group.d;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw nothing gives 0
      uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs;
      const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * S::kRows + half_row;
      float* part = p.part_o + at * p.part_dim;
      // 32 columns at a time, one copy of the code: unrolled, calls of few tokens took up to 0.7 us longer.
      // Of a shared item each warpgroup joins half of the columns.
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
      if (more && h == 1) load_queries(later);
      queries_loaded();
    }
    if (it.first && !it.last) {
      goes_on = true;
      if (threadIdx.x == 0) write_header(p, span, &it);
    }
    __syncwarp();  // every lane is done with the item
    if (lane == 0) it = later;
    __syncwarp();
    have = more;
  }
  cp_async_wait();  // of queries, after a wait that ran out
  if (threadIdx.x == 0 && !goes_on) write_header(p, span, nullptr);
}

template <int DT, int DP, int EXT>
__global__ void __launch_bounds__(kThreads, 1) attn_tma(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                        const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ SpanShared span;
  __shared__ Bars b;
  __shared__ SoftmaxState<DP> states[8];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // swizzled tiles start on 1024 bytes
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], 1);
      b.issued[i] = 0;
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(&b.s[x], 1);
      mbar_init(&b.o[x], 1);
      mbar_init(&b.p[x], 4);  // one arrival a warp
      mbar_init(&b.p2[x], 4);
    }
    for (int h = 0; h < 2; ++h) mbar_init(&b.q[h], 4);
    for (int x = 0; x < 2; ++x) mbar_init(&b.join[x], 8);
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

  const uint32_t queries = smem_addr(smem), ring = queries + S::kQueryBytes;
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      load_role<DP>(p, true, &kmap, span, b, ring);
    } else if (warp == kLoadWarp + 1) {
      load_role<DP>(p, false, &vmap, span, b, ring);
      check_blocks(p);
    } else if (warp == kMmaWarp) {
      mma_role<DT, DP>(p, span, b, queries, ring, tmem);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<DT, DP, EXT>(p, span, states[warp], b, smem, tmem);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (b.stop && warp == kLoadWarp)  // copies in flight end before the CTA does
    for (int i = 0; i < S::kSlots; ++i)
      if (b.issued[i] > (p.stall && i == 0 ? 1u : 0u)) mbar_wait_bounded(&b.full[i], (b.issued[i] - 1) & 1, p.wait_cycles);
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int DT, int DP>
const void* tma_of(int ext) {
  switch (ext) {
    case 0: return reinterpret_cast<const void*>(&attn_tma<DT, DP, 0>);
    case kCap: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kCap>);
    case kBias: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kBias>);
    case kCap | kBias | kWide: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kCap | kBias | kWide>);
    default: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kCap | kBias>);
  }
}

template <int DT>
const void* tma_of(int dp, int ext) {
  return dp == 64 ? tma_of<DT, 64>(ext) : dp == 128 ? tma_of<DT, 128>(ext) : tma_of<DT, 256>(ext);
}

}  // namespace

const void* attn_tma_kernel(bool bf16, int padded_dim, float cap, bool bias) {
  const int ext = score_forms(cap, bias);
  return bf16 ? tma_of<kBF16>(padded_dim, ext) : tma_of<kF16>(padded_dim, ext);
}

size_t attn_tma_smem(int padded_dim) {
  return (padded_dim == 64 ? Shape<64>::kBytes : padded_dim == 128 ? Shape<128>::kBytes : Shape<256>::kBytes) + 1024;
}

int attn_tma_rows(int padded_dim) { return padded_dim == 256 ? Shape<256>::kRows : Shape<128>::kRows; }

bool attn_tensor_map(void* encode, CUtensorMap* map, const void* base, CacheType type, int64_t dim, int64_t page, int64_t heads, int64_t blocks,
                     int64_t page_stride, int64_t head_stride, int64_t block_stride, int box_rows) {
  const int64_t es = type == CacheType::kE4M3 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)page, (cuuint64_t)heads, (cuuint64_t)blocks};
  // a dimension of one element has no stride to speak of
  const cuuint64_t strides[3] = {(cuuint64_t)(page > 1 ? page_stride * es : 16), (cuuint64_t)(heads > 1 ? head_stride * es : 16),
                                 (cuuint64_t)(blocks > 1 ? block_stride * es : 16)};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows, 1, 1}, steps[4] = {1, 1, 1, 1};
  // L2 fetches 256 bytes at a time only where they belong to the tile: rows of whole 256 bytes, or one
  // row right behind the other.  (64 requests' tokens over 350 MB, heads of 64 that lie between a token's
  // other heads: 141 us; with 256 bytes throughout 182 us.)
  const CUtensorMapL2promotion promotion =
      dim * es % 256 == 0 || page_stride == dim ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  const CUtensorMapDataType element = type == CacheType::kE4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : type == CacheType::kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  return reinterpret_cast<Encode>(encode)(map, element, 4, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                          CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ar

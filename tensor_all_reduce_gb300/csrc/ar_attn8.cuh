// What the attention kernels over a cache of E4M3 codes share: parts of 8 bits, the rings of keys, values and
// scales and the warps that fill them.
#pragma once

#include "ar_attn.cuh"
#include "ar_attn_tc.cuh"
#include "ar_e4m3.cuh"
#include "ar_staged.cuh"

namespace ar {

constexpr int kScaleTiles = 8;            // tiles of the ring of scales
constexpr int kScaleGroups = kKeys / 8;   // entries of a tile
constexpr int kUnitBytes = kKeys * 128;   // a ring slot: 128 rows of 128 codes

constexpr int kMostSlots = 4;

struct Ring {
  uint64_t full[kMostSlots], empty[kMostSlots];
  uint32_t issued[kMostSlots];  // rounds whose copies were issued, a slot
};

// ---- parts of 8 bits ----------------------------------------------------------

// Four floats -> four codes (E4M3 or E5M2), round to nearest even, saturating.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  if constexpr (E5M2)
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e5m2x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// What four E4M3 codes leave of four floats: exact, the codes being their roundings.
__device__ __forceinline__ void minus_codes4(uint32_t codes, float& a, float& b, float& c, float& d) {
  asm("{\n\t.reg .b16 x, y, lo, hi, one;\n\t.reg .b32 f, g;\n\tmov.b32 {x, y}, %4;\n\tmov.b16 one, 0xbc00;\n\t"
      "cvt.rn.f16x2.e4m3x2 f, x;\n\tcvt.rn.f16x2.e4m3x2 g, y;\n\t"
      "mov.b32 {lo, hi}, f;\n\tfma.rn.f32.f16 %0, lo, one, %0;\n\tfma.rn.f32.f16 %1, hi, one, %1;\n\t"
      "mov.b32 {lo, hi}, g;\n\tfma.rn.f32.f16 %2, lo, one, %2;\n\tfma.rn.f32.f16 %3, hi, one, %3;\n\t}"
      : "+f"(a), "+f"(b), "+f"(c), "+f"(d)
      : "r"(codes));
}

template <int PARTS>
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t (&part)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS - 1; ++i) {
    part[i] = codes4<false>(a, b, c, d);
    minus_codes4(part[i], a, b, c, d);
  }
  part[PARTS - 1] = codes4<true>(a, b, c, d);
}

// ---- tcgen05 --------------------------------------------------------------------

__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_count(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void sts_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// After tmem_wait_ld: keeps the uses of loaded registers behind the wait.
__device__ __forceinline__ void settle16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// ---- roles --------------------------------------------------------------------

// Keys or values, box by box through the block table: the lanes look the blocks up, one elected lane issues.
// (S: rows of an item and units of a tile; B: the barriers of a kernel, with its `stop`.)
template <class S, class B>
__device__ void load_role(const AttnParams& p, const CUtensorMap* map, const SpanShared& span, B& b, Ring& ring, uint32_t slots, uint32_t base, bool stall) {
  const int lane = threadIdx.x & 31;
  const int boxes = kKeys / p.box_rows;
  const bool one = elect_one();
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t n = 0, slot = 0, round = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    int block = 0, place = 0;  // block of this lane's box, and its place in the block
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
      // outside the cache: the copy fills with zeros
      const int w = (unsigned)block < (unsigned)p.num_blocks ? block : (int)p.num_blocks, y = place;
      if (t + 1 < nt) look_up(t + 1);
      for (int u = 0; u < S::kUnits; ++u, ++n) {
        ok = __all_sync(0xffffffffu, ok && wait_for(&ring.empty[slot], (round & 1) ^ 1, b, p));
        if (!ok) break;
        if (one) {
          mbar_arrive_expect_tx(&ring.full[slot], kUnitBytes);
          ring.issued[slot] = round + 1;
        }
        const uint32_t dst = base + slot * kUnitBytes;
        for (int x = 0; x < boxes; ++x) {
          const int wx = __shfl_sync(0xffffffffu, w, x), yx = __shfl_sync(0xffffffffu, y, x);
          if (one && !(stall && n == 0)) tma_4d(dst + x * p.box_rows * 128, map, u * 128, yx, it.h, wx, &ring.full[slot]);
        }
        if (++slot == slots) {
          slot = 0;
          ++round;
        }
      }
    }
  }
}

// The scales of two tiles at a time, a lane eight keys: the next blocks are looked up while the scales arrive.
template <class S, class B>
__device__ void scale_role(const AttnParams& p, const SpanShared& span, B& b, float4 (*ring)[kScaleGroups]) {
  const int lane = threadIdx.x & 31, second = lane >> 4, group = lane & 15;
  Walk<S::kRows, kKeys> walk;
  walk.start(span);
  Item it = {};
  uint32_t tiles = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    const int nt = it.end - it.begin;
    auto block_at = [&](int t) {  // -1: none, or outside the cache, which reads as zeros
      int block = -1;
      if (t + second < nt) {
        const int key = it.range.tile(it.begin + t + second) * kKeys + group * 8;
        if (key < it.q.len) block = p.table[(int64_t)it.r * p.table_stride + key / p.page];
      }
      return (unsigned)block < (unsigned)p.num_blocks ? block : -1;
    };
    int block = block_at(0);
    for (int t = 0; ok && t < nt; t += 2) {
      float4 v = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
      if (block >= 0) v = load_scales(p, block, it.h);
      block = block_at(t + 2);
      const uint32_t c = tiles + t, c1 = c + 1;
      const bool two = t + 1 < nt;
      ok = wait_for(&b.sc_empty[c % kScaleTiles], ((c / kScaleTiles) & 1) ^ 1, b, p) &&
           (!two || wait_for(&b.sc_empty[c1 % kScaleTiles], ((c1 / kScaleTiles) & 1) ^ 1, b, p));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (t + second < nt) ring[(c + second) % kScaleTiles][group] = v;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b.sc_full[c % kScaleTiles]);
        if (two) mbar_arrive(&b.sc_full[c1 % kScaleTiles]);
      }
    }
    tiles += nt;
  }
}

}  // namespace ar

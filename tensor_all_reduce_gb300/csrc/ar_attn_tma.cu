// Paged attention on the fifth-generation tensor cores: heads of up to 128 elements, rows on
// 16-byte boundaries, pages of a multiple of 8 tokens.
//
// A CTA (one an SM, resident) takes items of 256 query rows, two halves of 128, against tiles of
// 128 keys.  Of its twelve warps one loads keys and values by TMA, box by box through the block table,
// into a ring of shared-memory slots; one issues the matrix instructions; a warpgroup for each half
// turns scores into weights (the last two warps only complete the third warpgroup, which hands
// registers to the others).  A thread of a warpgroup owns one query row, so row maxima and
// sums need no exchange between threads.
//
// Tensor memory (512 columns of 128 lanes): scores of half h in columns [128 h, 128 h + 128), the
// weighted sum of half h in [256 + 128 h, ...).  The weights, 16-bit, take the first 64 columns
// of their half's scores and are the second product's A operand from there, so they never
// touch shared memory.  Matrix instructions of one CTA run in the order in which they are issued:
// while one half's softmax runs, the tensor core works on the other half's two products.
//
// The running maximum that the weights refer to moves only when a row's maximum has grown by more
// than 2^8 (in weight), since the result does not depend on the reference: then the sum in
// tensor memory is scaled.  Weights are thus at most 2^8, far inside both 16-bit ranges.
//
// Every wait is bounded; one that runs out leaves code 1 in the status word, and all roles stop.
#include <cuda.h>

#include "ar_attn.cuh"
#include "ar_staged.cuh"

namespace ar {
namespace {

constexpr int kRows = 256, kKeys = 128, kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr uint32_t kTmemCols = 512;
// 384 threads at 168 registers; the third warpgroup gives 96 a thread to the other two
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * 168, "the split uses what the launch has");

template <int DP>
struct Shape {
  static constexpr int kBlocks = DP / 64;               // 64-element (128-byte) column blocks of a row
  static constexpr int kBlockBytes = kKeys * 128;       // one column block of 128 rows
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kSlots = DP == 64 ? 10 : 5;
  static constexpr int kBytes = (2 + kSlots) * kTileBytes;
};

struct Bars {
  uint64_t full[10], empty[10];  // ring slots
  uint64_t q[2];                 // queries of a half stored
  uint64_t s[2];                 // scores of a half ready
  uint64_t p[2];                 // weights of a half stored
  uint64_t o[2];                 // sum of a half complete
  uint64_t drain;
  uint32_t tmem;
  int stop;
};

// ---- tcgen05 ----------------------------------------------------------------

__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// After tmem_wait_ld: keeps the uses of loaded registers behind the wait.
__device__ __forceinline__ void settle(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

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

// Arrives on `bar` when every matrix instruction this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes in groups of eight
// (1024 bytes apart).  `lead`: bytes between column blocks, for operands whose rows run along
// the reduction (values: a row is a key).
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: 16-bit operands, fp32 accumulator, 128 rows, n columns.
template <int DT>
__device__ __forceinline__ uint32_t instr_desc(int n, bool b_rows_along_k) {
  constexpr uint32_t type = DT == kBF16 ? 1 : 0;
  return (1u << 4) | (type << 7) | (type << 10) | ((b_rows_along_k ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// ---- two floats at a time -----------------------------------------------------

__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void untwo(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- waits --------------------------------------------------------------------

// Until the phase with `parity` completes; false when the wait ran out here or in another role.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Bars& b, const AttnParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&b.stop)) return false;
    if (clock64() - t0 > p.wait_cycles) {
      *reinterpret_cast<volatile int*>(&b.stop) = 1;
      *p.status = 1;
      return false;
    }
  }
  return true;
}

// ---- roles --------------------------------------------------------------------

using Steps = Walk<kRows, kKeys>;

__device__ __forceinline__ int halves(const Item& it) { return it.rows - it.qt * kRows > 128 ? 2 : 1; }

template <int DP>
__device__ void load_role(const AttnParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap, const SpanShared& span, Bars& b, uint32_t ring) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  const int boxes = kKeys / p.box_rows;
  const int box = lane / S::kBlocks, cb = lane - box * S::kBlocks;
  const bool issues = box < boxes;
  Steps walk(p, span);
  Item it;
  uint32_t n = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    for (int ti = it.begin; ok && ti < it.end; ++ti) {
      const int key = it.range.tile(ti) * kKeys + box * p.box_rows;
      int block = -1, in_page = 0;
      if (issues && key < it.q.len) block = (int)block_of(p, it.r, key, in_page);
      const int w = block < 0 ? (int)p.num_blocks : block;  // outside the cache: the copy fills with zeros
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t slot = n % S::kSlots, round = n / S::kSlots;
        ok = __all_sync(0xffffffffu, ok && wait_for(&b.empty[slot], (round & 1) ^ 1, b, p));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&b.full[slot], S::kTileBytes);
        __syncwarp();
        if (issues && !(p.stall && n == 0))
          tma_4d(ring + slot * S::kTileBytes + cb * S::kBlockBytes + box * p.box_rows * 128, kv ? vmap : kmap, cb * 64, in_page, it.h, w, &b.full[slot]);
        ++n;
      }
    }
  }
  if (!ok) {  // copies in flight end before the CTA does
    for (uint32_t i = n > S::kSlots ? n - S::kSlots : 0; i < n; ++i)
      if (!(p.stall && i == 0)) mbar_wait_bounded(&b.full[i % S::kSlots], (i / S::kSlots) & 1, p.wait_cycles);
  }
}

template <int DT, int DP>
__device__ void mma_role(const AttnParams& p, const SpanShared& span, Bars& b, uint32_t queries, uint32_t ring, uint32_t tmem) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  const int ksteps = (p.head_dim + 15) / 16;
  const uint32_t idesc_s = instr_desc<DT>(kKeys, false), idesc_o = instr_desc<DT>(ksteps * 16, true);
  // descriptors differ in the address alone, in units of 16 bytes: constant offsets are added
  const uint64_t q_desc = matrix_desc(queries, 16), k_desc = matrix_desc(ring, 16), v_desc = matrix_desc(ring, S::kBlockBytes);
  auto scores = [&](int h, uint32_t slot) {  // queries of half h times the keys in `slot`
    const uint64_t a = q_desc + h * (S::kTileBytes >> 4), k = k_desc + slot * (S::kTileBytes >> 4);
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const uint64_t off = ((i >> 2) * S::kBlockBytes + (i & 3) * 32) >> 4;
      if (i < ksteps) mma_ss(tmem + h * 128, a + off, k + off, idesc_s, i > 0);
    }
    mma_commit(&b.s[h]);
  };
  auto weighted = [&](int h, uint32_t slot, bool more) {  // weights of half h times the values in `slot`
    const uint64_t v = v_desc + slot * (S::kTileBytes >> 4);
#pragma unroll
    for (int i = 0; i < kKeys / 16; ++i)
      mma_ts(tmem + 256 + h * 128, tmem + h * 128 + i * 8, v + ((i * 16 * 128) >> 4), idesc_o, more || i > 0);
  };
  const bool one = elect_one();
  Steps walk(p, span);
  Item it;
  uint32_t n = 0, items[2] = {0, 0}, tiles[2] = {0, 0};
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait_for(bar, parity, b, p));
    fence_after();
    return ok;
  };
  while (ok && walk.next(p, it)) {
    const int nh = halves(it), nt = it.end - it.begin;
    uint32_t slot = n % S::kSlots;
    if (!wait(&b.full[slot], (n / S::kSlots) & 1)) break;
    for (int h = 0; h < nh; ++h) {
      if (!wait(&b.q[h], items[h]++ & 1)) break;
      if (one) scores(h, slot);
    }
    if (!ok) break;
    if (one) mma_commit(&b.empty[slot]);
    ++n;
    for (int i = 0; ok && i < nt; ++i) {
      const uint32_t vs = n % S::kSlots, ks = (n + 1) % S::kSlots;
      const bool more = i + 1 < nt;
      if (!wait(&b.full[vs], (n / S::kSlots) & 1)) break;
      const int key0 = it.range.tile(it.begin + i) * kKeys, left = it.q.len - key0;
      if (left < kKeys) {
        // values behind the request's end: whole boxes came as zeros, the rest of the last
        // box holds whatever the cache does
        const int lo = max(left, 0), hi = min((lo + p.box_rows - 1) / p.box_rows * p.box_rows, kKeys);
        const uint32_t v = ring + vs * S::kTileBytes;
        for (int x = lo * 8 + lane; x < hi * 8; x += 32)
#pragma unroll
          for (int cb = 0; cb < S::kBlocks; ++cb)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + cb * S::kBlockBytes + x * 16), "r"(0) : "memory");
        fence_proxy_async_smem();
        __syncwarp();
      }
      for (int h = 0; h < nh; ++h) {
        if (!wait(&b.p[h], tiles[h]++ & 1)) break;
        if (one) weighted(h, vs, i > 0);
        if (more) {
          if (h == 0 && !wait(&b.full[ks], ((n + 1) / S::kSlots) & 1)) break;
          if (one) scores(h, ks);
        } else if (one) {
          mma_commit(&b.o[h]);
        }
      }
      if (!ok) break;
      if (one) {
        mma_commit(&b.empty[vs]);
        if (more) mma_commit(&b.empty[ks]);
      }
      n += more ? 2 : 1;
    }
  }
  if (!ok) {  // matrix instructions in flight end before tensor memory is freed
    if (one) mma_commit(&b.drain);
    mbar_wait_bounded(&b.drain, 0, p.wait_cycles);
  }
}

// How scores are bent, a bit each: kCap (tanh), kBias (distance; also any scale that is not positive,
// since the plain form scales after the maximum).
enum { kCap = 1, kBias = 2 };

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's products over the tile's 128 keys to scores, masked: in log2 units where they are
// bent, else as they are (the caller scales).
template <int EXT>
__device__ __forceinline__ void shape_scores(const AttnParams& p, const Item& it, const RowView& v, int key0, float (&s)[kKeys]) {
  if constexpr (EXT & kCap) {
    // c tanh(x) = c - 2 c / (1 + e^2x): one exponential and one reciprocal an element, absolute
    // error 2^-22 c; an exponential that overflows gives c
    const float twice = p.scale_log2 * 2.8853900817779268f, c = p.cap_log2;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) s[j] = fmaf(-2.0f * c, rcp(1.0f + ex2(s[j] * twice)), c);
  }
  if constexpr (EXT & kBias) {
    const float scale = EXT & kCap ? 1.0f : p.scale_log2;
    const float far = (float)(v.pos - key0);
#pragma unroll
    for (int j = 0; j < kKeys; ++j) s[j] = fmaf(-v.slope, fabsf(far - (float)j), s[j] * scale);
  }
  // the whole warp sees the whole tile: nothing to mask
  const bool all = (key0 + kKeys <= v.see_hi && key0 >= v.see_lo) || key0 + kKeys <= it.q.prefix;
  if (__all_sync(0xffffffffu, all)) return;
  const int hi = v.see_hi - key0, lo = v.see_lo - key0, pre = it.q.prefix - key0;
#pragma unroll
  for (int j = 0; j < kKeys; ++j)
    if (!(j < pre || (j < hi && j >= lo))) s[j] = -INFINITY;
}

template <int DT, int DP, int EXT>
__device__ void softmax_role(const AttnParams& p, const SpanShared& span, Bars& b, uint8_t* queries, uint32_t tmem, bool (&wrote)[2]) {
  using S = Shape<DP>;
  const int h = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t ts = lanes + h * 128, to = lanes + 256 + h * 128;
  const float scale = EXT ? 1.0f : p.scale_log2;
  Steps walk(p, span);
  Item it;
  uint32_t items = 0, tiles = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    if (h >= halves(it)) continue;
    const int base_row = it.qt * kRows + h * 128;
    // queries, 16 bytes a thread, neighbours along a row; rows and columns beyond are zero
    uint8_t* dst = queries + h * S::kTileBytes;
#pragma unroll 4
    for (int x = tid; x < 128 * (DP / 8); x += 128) {
      const int r = x / (DP / 8), c = x % (DP / 8), row = base_row + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < it.rows && c * 8 < p.head_dim) {
        const int t = row / p.group, g = row - t * p.group;
        v = ld_keep(static_cast<const uint16_t*>(p.q) + (int64_t)(it.q.q0 + t) * p.q_ts + (int64_t)(it.h * p.group + g) * p.q_hs + c * 8);
      }
      *reinterpret_cast<uint4*>(dst + (c >> 3) * S::kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
    mbar_arrive(&b.q[h]);

    const int row = base_row + tid;
    const bool busy = base_row + warp * 32 < it.rows;  // the warp has a row
    RowView view = row_view(p, it, row);
    if (row >= it.rows) {  // no row: sees all, so that the warp need not mask for it; nothing of it is stored
      view.see_lo = 0;
      view.see_hi = 0x7fffffff;
    }
    float m = -INFINITY;
    uint64_t sum = two(0.0f, 0.0f);
    for (int ti = it.begin; ti < it.end; ++ti) {
      ok = wait_for(&b.s[h], tiles++ & 1, b, p);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      fence_after();
      if (busy) {
        uint32_t raw[kKeys / 32][32];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(raw[c], ts + c * 32);
        tmem_wait_ld();
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) {
          settle(raw[c]);
#pragma unroll
          for (int j = 0; j < 32; ++j) s[c * 32 + j] = __uint_as_float(raw[c][j]);
        }
        shape_scores<EXT>(p, it, view, it.range.tile(ti) * kKeys, s);
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < kKeys; ++j) top[j & 3] = fmaxf(top[j & 3], s[j]);
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
        const bool grown = high > m + 8.0f;  // m = -inf: any finite score
        if (__any_sync(0xffffffffu, grown)) {
          const float shrink = grown ? ex2(m - high) : 1.0f;  // m = -inf: 0
          if (grown) m = high;
          if (ti > it.begin) {
            float lo, hi;
            untwo(sum, lo, hi);
            sum = two(lo * shrink, hi * shrink);
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o, to + c * 32);
              tmem_wait_ld();
              settle(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
              tmem_st32(to + c * 32, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        const uint64_t scale2 = two(scale, scale), base2 = two(-base, -base);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int e = c * 64 + j * 2;
            float a, z;
            untwo(fma2(two(s[e], s[e + 1]), scale2, base2), a, z);
            a = ex2(a);
            z = ex2(z);
            sum = add2(sum, two(a, z));  // of the unrounded weights
            w[j] = pack2<DT>(a, z);      // the second product's operand is 16-bit: half a step, relative, a weight
          }
          tmem_st32(ts + c * 32, w);
        }
        tmem_wait_st();
      }
      fence_before();
      mbar_arrive(&b.p[h]);
    }
    if (!ok) break;
    ok = __all_sync(0xffffffffu, wait_for(&b.o[h], items++ & 1, b, p));
    if (!ok) break;
    fence_after();
    const bool whole = it.first && it.last;
    const int slot = it.first ? 1 : 0;
    if (busy) {
      float lo, hi;
      untwo(sum, lo, hi);
      const float l = lo + hi;
      const bool mine = row < it.rows;
      const int t = row / p.group, head = it.h * p.group + row - t * p.group;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)(it.q.q0 + t) * p.o_ts + (int64_t)head * p.o_hs;
      const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * kRows + h * 128 + tid;
      float* part = p.part_o + at * p.part_dim;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o, to + c * 32);
        tmem_wait_ld();
        settle(o);
        if (!mine) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          if (c * 32 + j >= p.head_dim) break;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[j + e]);
          if (whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = l > 0.0f ? f[e] * inv : 0.0f;
            st_v4(out + c * 32 + j, pack8<DT>(f));
          } else {
            *reinterpret_cast<float4*>(part + c * 32 + j) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(part + c * 32 + j + 4) = make_float4(f[4], f[5], f[6], f[7]);
          }
        }
      }
      if (mine && whole && p.lse) p.lse[(int64_t)(it.q.q0 + t) * p.q_heads + head] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      if (mine && !whole) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
    }
    if (!whole) {
      wrote[slot] = true;
      if (threadIdx.x == 0) write_header(p, slot, kThere | (it.last ? kEnds : 0), &it);
    }
    fence_before();
  }
}

template <int DT, int DP, int EXT>
__global__ void __launch_bounds__(kThreads, 1) attn_tma(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                        const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ SpanShared span;
  __shared__ Bars b;
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // swizzled tiles start on 1024 bytes
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&b.q[h], 128);
      mbar_init(&b.s[h], 1);
      mbar_init(&b.p[h], 128);
      mbar_init(&b.o[h], 1);
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
  find_span<kRows, kKeys, kThreads>(p, span);

  const uint32_t queries = smem_addr(smem), ring = queries + 2 * S::kTileBytes;
  bool wrote[2] = {false, false};
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp)
      load_role<DP>(p, &kmap, &vmap, span, b, ring);
    else if (warp == kMmaWarp)
      mma_role<DT, DP>(p, span, b, queries, ring, tmem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<DT, DP, EXT>(p, span, b, smem, tmem, wrote);
  }
  if (threadIdx.x == 0)
    for (int s = 0; s < 2; ++s)
      if (!wrote[s]) write_header(p, s, 0, nullptr);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int DT, int DP>
const void* tma_of(int ext) {
  switch (ext) {
    case 0: return reinterpret_cast<const void*>(&attn_tma<DT, DP, 0>);
    case kCap: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kCap>);
    case kBias: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kBias>);
    default: return reinterpret_cast<const void*>(&attn_tma<DT, DP, kCap | kBias>);
  }
}

template <int DT>
const void* tma_of(int dp, int ext) {
  return dp == 64 ? tma_of<DT, 64>(ext) : tma_of<DT, 128>(ext);
}

}  // namespace

const void* attn_tma_kernel(bool bf16, int padded_dim, bool cap, bool bias) {
  const int ext = (cap ? kCap : 0) | (bias ? kBias : 0);
  return bf16 ? tma_of<kBF16>(padded_dim, ext) : tma_of<kF16>(padded_dim, ext);
}

size_t attn_tma_smem(int padded_dim) { return (padded_dim == 64 ? Shape<64>::kBytes : Shape<128>::kBytes) + 1024; }

bool attn_tensor_map(void* encode, CUtensorMap* map, const void* base, bool bf16, int64_t dim, int64_t page, int64_t heads, int64_t blocks,
                     int64_t page_stride, int64_t head_stride, int64_t block_stride, int box_rows) {
  const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)page, (cuuint64_t)heads, (cuuint64_t)blocks};
  // a dimension of one element has no stride to speak of
  const cuuint64_t strides[3] = {(cuuint64_t)(page > 1 ? page_stride * 2 : 16), (cuuint64_t)(heads > 1 ? head_stride * 2 : 16),
                                 (cuuint64_t)(blocks > 1 ? block_stride * 2 : 16)};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, steps[4] = {1, 1, 1, 1};
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  return reinterpret_cast<Encode>(encode)(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                                          const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ar
